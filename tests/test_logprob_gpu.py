"""Log probabilities of given tokens, entropy, top alternatives and their
gradient against the definitions in 64 bits.

Tolerances, with u = 2^-24.  d = (l - m) / T in units of ln 2 takes a
difference, a product and a factor that itself carries three roundings:
within 6 u of itself, so exp(d) is within (4 + 6 |d|) u relative (d natural;
the power of two's own error is at most 2^-22).  S adds these in chains of at
most V / 512 + 48 additions per thread and 60 more with the rescalings and
joins: its relative error is at most
    eS = (4 + 6 sum p |d| + V / 512 + 108) u,
which is also the error of log S beside its own roundings.  U = sum e d is
off by eS and by 6 u of sum p d^2.  What follows from these is written at
each check.
"""
import math

import pytest
import torch

import row_normalization_inner_gb300 as nf

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    yield


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make(rows, vocab, kind, fill, seed, room=0, shift=0):
    """Logits, possibly as rows `room` elements longer than the vocabulary that start `shift` elements in."""
    g = gen(seed)
    full = torch.full((rows, vocab + room + shift), 77.0, device="cuda", dtype=TYPES[kind])
    l = torch.randn(rows, vocab, generator=g, device="cuda") * 3
    if fill == "equal":
        l[:] = 1.5
    elif fill == "rising":
        l = torch.arange(vocab, device="cuda").float().repeat(rows, 1) / max(vocab, 1) * 20 - 5
    elif fill == "peak":
        l.scatter_(1, torch.randint(0, vocab, (rows, 1), generator=g, device="cuda"), 40.0)
    elif fill == "masked":
        l.masked_fill_(torch.rand(rows, vocab, generator=g, device="cuda") < 0.6, -math.inf)
        l[-1] = -math.inf
    elif fill == "nearly masked":
        l[:] = -math.inf
        l[:, vocab // 2] = 2.0
    elif fill == "lowest":
        l.masked_fill_(torch.rand(rows, vocab, generator=g, device="cuda") < 0.6, torch.finfo(TYPES[kind]).min)
        l[-1] = torch.finfo(TYPES[kind]).min
    full[:, shift:shift + vocab] = l.to(TYPES[kind])
    targets = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    return full[:, shift:shift + vocab], targets


class Ref:
    """The definitions in 64 bits."""

    def __init__(self, logits, targets, temperature):
        inv = 1.0 / torch.tensor(temperature, dtype=torch.float32).double().item()
        l = logits.double()
        rows, vocab = l.shape
        self.m = l.amax(1)
        self.empty = self.m == -math.inf
        d = (l - torch.where(self.empty, 0.0, self.m)[:, None]) * inv
        e = d.exp()
        s = e.sum(1)
        self.log_s = s.log()
        self.d, self.p = d, torch.where(self.empty[:, None], 0.0, e / s[:, None])
        dz = torch.where(e > 0, d, 0.0)
        self.mean_d = torch.where(self.empty, 0.0, (self.p * dz).sum(1))       # <= 0
        self.mean_d2 = torch.where(self.empty, 0.0, (self.p * dz * dz).sum(1))
        self.entropy = torch.where(self.empty, 0.0, self.log_s - self.mean_d)
        known = (targets >= 0) & (targets < vocab)
        self.at = targets.long().clamp(0, vocab - 1)
        self.known = known
        lp = d.gather(1, self.at[:, None])[:, 0] - self.log_s
        lp = torch.where(self.empty, -math.inf, lp)
        self.logprob = torch.where(known, lp, 0.0)
        self.err_s = (4 - 6 * self.mean_d + vocab / 512 + 108) * U
        self.inv = inv


def close(got, want, tol):
    """Equal where infinite, within tol where finite.  What lies beyond fp32's
    largest value (the type's lowest number as a mask, at a temperature below
    1) is infinite in fp32."""
    want = torch.where(want.abs() > torch.finfo(torch.float32).max, want.float().double(), want)
    fin = want.isfinite()
    assert torch.equal(got.double()[~fin], want[~fin])
    assert torch.all(((got.double() - want).abs() <= tol)[fin]), ((got.double() - want).abs() / tol)[fin].max()


def check_forward(logits, targets, temperature, top):
    logprob, entropy, stats, top_lp, top_ids = nf.token_logprob_fwd(logits, targets, temperature, top=top)
    r = Ref(logits, targets, temperature)
    log_s = torch.where(r.empty, 0.0, r.log_s)
    err_log = r.err_s + 3 * U * log_s.abs()
    d_t = torch.where(r.empty, 0.0, r.d.gather(1, r.at[:, None])[:, 0])
    close(logprob, r.logprob, err_log + 6 * U * d_t.abs() + U * r.logprob.abs())
    close(entropy, r.entropy, err_log + 2 * r.err_s * r.mean_d.abs() + 6 * U * r.mean_d2 + 4 * U * (log_s + r.mean_d.abs()))
    assert torch.equal(stats[:, 0].double(), r.m)
    close(stats[:, 1], r.log_s, err_log)
    if not top:
        assert top_lp is None and top_ids is None
        return logprob, entropy, stats
    vocab = logits.shape[1]
    best, ids = torch.sort(logits.double(), dim=1, descending=True, stable=True)
    want_ids = torch.full((len(logits), top), -1, device="cuda")
    want_lp = torch.full((len(logits), top), -math.inf, dtype=torch.float64, device="cuda")
    k = min(top, vocab)
    want_ids[:, :k] = torch.where(best[:, :k] > -math.inf, ids[:, :k], -1)
    d = (best[:, :k] - torch.where(r.empty, 0.0, r.m)[:, None]) * r.inv
    want_lp[:, :k] = torch.where(best[:, :k] > -math.inf, d - log_s[:, None], -math.inf)
    assert torch.equal(top_ids, want_ids)
    d = torch.where(want_lp.isfinite(), want_lp + log_s[:, None], 0.0)
    close(top_lp, want_lp, err_log[:, None] + 6 * U * d.abs() + U * want_lp.abs())
    return logprob, entropy, stats


SIZES = [(1, 1), (3, 2), (2, 7), (5, 31), (300, 128), (4, 1000), (700, 1001), (16, 4097), (1, 32003), (310, 32003),
         (2, 100003), (16, 131072), (40, 65536), (160, 70001)]
FILLS = ["normal", "equal", "rising", "peak", "masked", "nearly masked", "lowest"]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_forward(rows, vocab, fill, kind):
    logits, targets = make(rows, vocab, kind, fill, rows + vocab)
    for top, temperature in ((0, 1.0), (1, 0.5), (5, 1.0), (32, 1.7)):
        check_forward(logits, targets, temperature, top)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("rows,vocab", [(1600, 7), (1601, 1000), (1533, 4097), (1520, 9001), (1521, 20011)])
def test_forward_of_many_rows(rows, vocab, fill, kind):
    logits, targets = make(rows, vocab, kind, fill, rows + vocab, room=3, shift=1)
    for top, temperature in ((0, 1.0), (32, 0.7)):
        check_forward(logits, targets, temperature, top)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shift,room", [(1, 0), (3, 5), (0, 13), (8, 8), (7, 9)])
@pytest.mark.parametrize("rows,vocab", [(3, 5), (9, 1000), (20, 33000), (400, 2049)])
def test_forward_rows_that_start_anywhere(rows, vocab, shift, room, kind):
    logits, targets = make(rows, vocab, kind, "normal", vocab, room=room, shift=shift)
    check_forward(logits, targets.int(), 0.9, 20)


def test_top_of_rows_whose_best_share_a_thread():
    # the largest values 4096 apart: the same lanes hold many of them
    for kind in ("bf16", "f32"):
        logits, targets = make(4, 131072, kind, "normal", 1)
        logits[:, 5::4096] = torch.arange(32, device="cuda").to(logits.dtype) + 20
        logits[1, 5::2048] = 30.0
        logits[2, ::2] = 31.0
        check_forward(logits, targets, 1.0, 32)


def zeros_of_both_signs(rows, vocab, kind, layout):
    """Logits whose largest entries are zeros of both signs, everything else below -1."""
    g = gen(vocab + len(layout))
    l = -1 - torch.rand(rows, vocab, generator=g, device="cuda") * 5
    sign = torch.where(torch.rand(rows, vocab, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    col = torch.arange(vocab, device="cuda")
    if layout == "few":          # about 40 a row: the border of 32 alternatives lies among them
        l = torch.where(torch.rand(rows, vocab, generator=g, device="cuda") < 40 / vocab, 0.0 * sign, l)
    elif layout == "all":
        l = 0.0 * sign
    elif layout == "rising":     # -0 at the lower ids: a thread's first batches, the first CTAs of a cluster
        l = torch.where(col % 3 == 0, torch.where(col < vocab // 2, -0.0, 0.0), l)
    elif layout == "falling":
        l = torch.where(col % 3 == 0, torch.where(col < vocab // 2, 0.0, -0.0), l)
    elif layout == "one of +0":  # -0 wherever a thread looks, one +0 behind
        l = torch.where(col % 2 == 0, -0.0, l)
        l[:, vocab - 1 - vocab // 5] = 0.0
    return l.to(TYPES[kind])


# one batch per thread, several, a cluster per row, and small CTAs of many rows
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["few", "all", "rising", "falling", "one of +0"])
@pytest.mark.parametrize("rows,vocab", [(3, 2), (4, 39), (5, 1000), (16, 4097), (2, 131072), (310, 32003), (400, 32003),
                                        (1601, 1000), (1533, 9001)])
def test_zeros_of_both_signs_are_equal(rows, vocab, layout, kind):
    logits = zeros_of_both_signs(rows, vocab, kind, layout)
    targets = torch.zeros(rows, dtype=torch.int64, device="cuda")
    values = logits.double() + 0.0  # -0 becomes +0: ties by id alone
    best, order = torch.sort(values, dim=1, descending=True, stable=True)
    for top in (1, 5, 32):
        _, _, stats, top_lp, top_ids = nf.token_logprob_fwd(logits, targets, 1.0, top=top)
        k = min(top, vocab)
        assert torch.equal(top_ids[:, :k], order[:, :k])
        assert torch.all(top_ids[:, k:] == -1)
        # equal logits have equal log probabilities, whatever the zero's sign: m - m - log S
        zero = best[:, :k] == 0
        assert torch.equal(top_lp[:, :k][zero], (-stats[:, 1:]).expand(rows, k)[zero])


@pytest.mark.parametrize("rows", [2, 400])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_with_nan_and_infinity(kind, rows):
    logits, targets = make(rows, 5000, kind, "normal", 3)
    logits[0, 1234] = float("nan")
    logits[1, 4999] = float("inf")
    logprob, entropy, stats, top_lp, top_ids = nf.token_logprob_fwd(logits, targets, top=4)
    for r in (0, 1):
        assert torch.isnan(logprob[r]) and torch.isnan(entropy[r]) and torch.isnan(stats[r, 1])
        assert torch.isnan(top_lp[r]).all() and torch.all(top_ids[r] == -1)
    if rows > 2:
        check_forward(logits[2:], targets[2:], 1.0, 4)
    out = nf.token_logprob_bwd(logits, targets, stats, entropy, torch.ones(rows, device="cuda"))
    assert torch.isnan(out[:2]).all() and torch.isfinite(out[2:]).all()


def test_targets_outside_the_vocabulary():
    logits, _ = make(6, 3000, "f32", "normal", 4)
    logits[4:] = -math.inf
    targets = torch.tensor([-1, 3000, 1 << 40, -100, -1, 7], device="cuda")
    logprob, entropy, stats = check_forward(logits, targets, 1.0, 0)
    assert torch.all(logprob[:5] == 0) and logprob[5] == -math.inf
    assert torch.all(entropy[:4] > 0) and torch.all(entropy[4:] == 0)
    g = torch.ones(6, device="cuda")
    assert torch.all(nf.token_logprob_bwd(logits, targets, stats, entropy, g) == 0)
    check_gradient(logits, targets, 1.0, True)


# ---------------------------------------------------------------- gradient

def check_gradient(logits, targets, temperature, with_entropy, out=None):
    rows, vocab = logits.shape
    r = Ref(logits, targets, temperature)
    stats = torch.stack([r.m, r.log_s], 1).float()
    entropy = r.entropy.float()
    g = torch.randn(rows, generator=gen(rows), device="cuda")
    h = torch.randn(rows, generator=gen(vocab), device="cuda") if with_entropy else None
    got = nf.token_logprob_bwd(logits, targets, stats, entropy if with_entropy else None, g, h, temperature, out=out)
    assert got.shape == logits.shape and got.dtype == logits.dtype
    gd = torch.where(r.known & ~r.empty, g.double(), 0.0)[:, None]
    hd = (torch.zeros_like(g) if h is None else h).double()[:, None]
    log_s = torch.where(r.empty, 0.0, r.log_s)[:, None]
    log_p = torch.where(r.p > 0, r.d - log_s, 0.0)
    ent = r.entropy[:, None]
    ref = -gd * r.p - hd * r.p * (log_p + ent)
    ref.scatter_add_(1, r.at[:, None], gd)
    ref = ref * r.inv
    # log p is off by 6 u |d| and 4 u |log S| (the fp32 stats, and two differences), p by that and 4 u;
    # the factor A + B log p by 6 u of its parts' sizes and by log p's error; a p below fp32's smallest
    # normal number, 2^-126, is 0
    e_log = 6 * U * torch.where(r.p > 0, r.d, 0.0).abs() + 4 * U * log_s.abs() + 2 * U * log_p.abs()
    parts = gd.abs() + hd.abs() * (ent.abs() + log_p.abs())
    tol = r.inv * (r.p * (parts * (e_log + 14 * U) + hd.abs() * e_log) + torch.clamp(r.p, max=2.0 ** -126) * parts)
    tol = tol + 3 * U * r.inv * torch.zeros_like(ref).scatter_add_(1, r.at[:, None], gd.abs()) + 1e-37
    if logits.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert torch.all((got.double() - ref).abs() <= tol), ((got.double() - ref).abs() / tol).max()
    return got


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_gradient(rows, vocab, fill, kind):
    logits, targets = make(rows, vocab, kind, fill, rows + vocab)
    check_gradient(logits, targets, 1.0, False)
    check_gradient(logits, targets, 0.6, True)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shift,room", [(0, 0), (1, 2), (0, 13), (8, 8)])
def test_gradient_in_place_strided_and_beside(shift, room, kind):
    rows, vocab = 50, 2049
    logits, targets = make(rows, vocab, kind, "normal", 6, room=room, shift=shift)
    want = check_gradient(logits, targets, 1.0, True)
    # rows of another alignment, with columns behind the vocabulary
    big = torch.full((rows, vocab + 6), 5.0, dtype=logits.dtype, device="cuda")
    got = check_gradient(logits, targets, 1.0, True, out=big[:, 3:3 + vocab])
    assert torch.equal(got, want)
    assert torch.all(big[:, :3] == 5) and torch.all(big[:, 3 + vocab:] == 5)
    # in place: what lies around the rows stays
    whole = logits.as_strided((rows, vocab + room + shift), logits.stride(), logits.storage_offset() - shift)
    got = check_gradient(logits, targets, 1.0, True, out=logits)
    assert got is logits and torch.equal(got, want)
    assert torch.all(whole[:, :shift] == 77) and torch.all(whole[:, shift + vocab:] == 77)


@pytest.mark.parametrize("kind,rows,vocab", [("bf16", 2503, 131072 + 5), ("f32", 3400, 50001)])
def test_gradient_of_large_calls(kind, rows, vocab):
    # several batches of a row per CTA; checked some rows at a time
    logits = torch.randn(rows, vocab, generator=gen(7), device="cuda").mul_(3).to(TYPES[kind])
    targets = torch.randint(0, vocab, (rows,), generator=gen(8), device="cuda")
    g = torch.randn(rows, generator=gen(9), device="cuda")
    h = torch.randn(rows, generator=gen(10), device="cuda")
    _, ent, stats, _, _ = nf.token_logprob_fwd(logits, targets)
    got = nf.token_logprob_bwd(logits, targets, stats, ent, g, h)
    for at in (0, 1, 97, rows // 2, rows - 3):
        part = slice(at, at + 3)
        want = nf.token_logprob_bwd(logits[part], targets[part], stats[part], ent[part], g[part], h[part])
        assert torch.equal(got[part], want)
        check_gradient(logits[part], targets[part], 1.0, True)
    sums = got.float().sum(1)  # every row's gradient sums to 0
    assert torch.all(sums.abs() < 0.05 * (1 + g.abs() + h.abs()))


def test_gradient_against_differences():
    # central differences of the operator's own forward along random directions: with a step of 2^-6 the
    # third-order term is below (2^-6)^2 / 6 * 30 (third derivatives of log softmax and entropy along a unit
    # direction stay below 30 for |log p| < 25), and the forward's error of 4e-6 counts 4e-6 / 2^-6
    rows, vocab, h = 64, 400, 2.0 ** -6
    logits, targets = make(rows, vocab, "f32", "normal", 8)
    logits = logits.clone()
    g = torch.randn(rows, generator=gen(1), device="cuda")
    e = torch.randn(rows, generator=gen(2), device="cuda")
    lp, ent, stats, _, _ = nf.token_logprob_fwd(logits, targets, 0.8)
    grad = nf.token_logprob_bwd(logits, targets, stats, ent, g, e, 0.8)
    scale = (g.abs() + e.abs()) * 0.8 ** -3 * (h * h / 6 * 30 + 4e-6 / h)
    for seed in range(4):
        way = torch.randn(rows, vocab, generator=gen(10 + seed), device="cuda")
        way[:, 0] += 10
        way /= way.norm(dim=1, keepdim=True)
        up, down = (nf.token_logprob_fwd(logits + s * h * way, targets, 0.8)[:2] for s in (1, -1))
        diff = (g * (up[0] - down[0]) + e * (up[1] - down[1])) / (2 * h)
        assert torch.all((diff - (grad * way).sum(1)).abs() <= scale)


# ---------------------------------------------------------------- calls

def test_large_offsets():
    # rows beyond 2^31 elements
    rows, vocab = 17, 1 << 27
    logits = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    logits[-1, -1] = 30.0
    logits[-1, 3] = 31.0
    targets = torch.full((rows,), vocab - 1, device="cuda")
    lp, ent, stats, top_lp, top_ids = nf.token_logprob_fwd(logits, targets, top=2)
    assert top_ids[-1].tolist() == [3, vocab - 1] and top_ids[0].tolist() == [0, 1]
    s = math.log((vocab - 2) * math.exp(-31.0) + math.exp(-1.0) + 1)
    assert abs(lp[-1].item() - (-1 - s)) < 1e-5
    assert abs(ent[0].item() - math.log(vocab)) < 1e-3
    out = nf.token_logprob_bwd(logits, targets, stats, ent, torch.ones(rows, device="cuda"), out=logits)
    assert abs(out[-1, -1].item() - (1 - math.exp(-1 - s))) < 2e-3
    assert abs(out[0, -1].item() - 1) < 1e-3 and out[0, 0].item() < 0


def test_deterministic_another_stream_and_graph():
    for rows, vocab in ((8, 50001), (400, 3000)):
        logits, targets = make(rows, vocab, "bf16", "normal", 5)
        want = nf.token_logprob_fwd(logits, targets, top=8)
        g = torch.ones(rows, device="cuda")
        grad = nf.token_logprob_bwd(logits, targets, want[2], want[1], g, g)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        got = nf.token_logprob_fwd(logits, targets, top=8, stream=side)
        got_grad = nf.token_logprob_bwd(logits, targets, got[2], got[1], g, g, stream=side)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(got_grad, grad)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = nf.token_logprob_fwd(logits, targets, top=8)
            got_grad = nf.token_logprob_bwd(logits, targets, got[2], got[1], g, g)
        for _ in range(3):
            for x in got:
                x.zero_()
            got_grad.zero_()
            graph.replay()
            assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(got_grad, grad)


def test_helper_refusals():
    logits, targets = make(4, 100, "bf16", "normal", 1)
    lp, ent, stats, _, _ = nf.token_logprob_fwd(logits, targets)
    empty = nf.token_logprob_fwd(logits[:0], targets[:0], top=3)
    assert empty[0].shape == (0,) and empty[4].shape == (0, 3)
    assert nf.token_logprob_bwd(logits[:0], targets[:0], stats[:0], ent[:0], lp[:0]).shape == (0, 100)
    for call in (lambda: nf.token_logprob_fwd(logits, targets[:3]), lambda: nf.token_logprob_fwd(logits[0], targets),
                 lambda: nf.token_logprob_fwd(logits.t(), targets), lambda: nf.token_logprob_fwd(logits, targets, top=33),
                 lambda: nf.token_logprob_fwd(logits[:, ::2], targets),
                 lambda: nf.token_logprob_fwd(logits[:1].expand(4, 100), targets),
                 lambda: nf.token_logprob_bwd(logits, targets, stats[:3], ent, lp),
                 lambda: nf.token_logprob_bwd(logits, targets, stats, ent[:3], lp, lp),
                 lambda: nf.token_logprob_bwd(logits, targets, stats, ent, lp, out=logits.float())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        nf.token_logprob_bwd(logits, targets, stats, ent, lp.double())
    with pytest.raises(nf.NFError):
        nf.token_logprob_fwd(logits, targets, 0.0)
    with pytest.raises(nf.NFError):
        nf.token_logprob_bwd(logits, targets, stats, ent, lp, temperature=-1.0)
