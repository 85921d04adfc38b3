"""The token-side operators together, as a model uses them: tokens to rows,
a normalized block, log probabilities, and back to the table's gradient;
and the serving side with 8-bit rows.

Tolerances.  Every stage rounds its output to bf16 (half a step: 2^-8), and
the stages are few and well conditioned, so gradients are compared in the
2-norm against a 64-bit evaluation of the same model: with R roundings to
bf16 on the way to a result, each off by at most 2^-8 of its own tensor and
independent of the others, the result is off by at most R * 2^-8 of its norm
times the gain of the stages behind it, which the normalization keeps near 1;
4 R * 2^-8 is asserted.
"""
import math

import pytest
import torch

import row_normalization_inner_gb300 as nf

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    yield


class Model:
    """table -> scaled rows -> residual add of a linear branch, RMSNorm -> tied output layer."""

    def __init__(self, tokens=640, vocab=2003, hidden=512, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def draw(*shape):
            return torch.randn(*shape, generator=g, device="cuda")
        self.tokens, self.vocab, self.hidden = tokens, vocab, hidden
        self.table = (draw(vocab, hidden) / math.sqrt(hidden)).bfloat16()
        self.branch = (draw(hidden, hidden) / math.sqrt(hidden)).bfloat16()
        self.w = (1 + 0.1 * draw(hidden)).bfloat16()
        self.ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        self.ids[::9] = 7          # one id that fills several chunks
        self.ids[5::31] = -1       # padding
        self.targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        self.targets[5::31] = -1
        self.scale = math.sqrt(hidden)
        self.d_logprob = draw(tokens)
        self.d_entropy = 0.1 * draw(tokens)

    def forward(self):
        self.x0 = nf.embedding_fwd(self.ids, self.table, self.scale)
        self.y = self.x0 @ self.branch
        self.res = self.x0.clone()
        nf.fused_add_rmsnorm(self.y, self.res, self.w, EPS)      # y: normalized rows, res: the stream
        self.logits = self.y @ self.table.t()
        self.logprob, self.entropy, self.stats, self.top, self.top_ids = nf.token_logprob_fwd(
            self.logits, self.targets, 1.0, top=4)
        return self.logprob, self.entropy

    def backward(self):
        """Gradient of sum(d_logprob * logprob + d_entropy * entropy) for the table and the norm's weight."""
        dlogits = nf.token_logprob_bwd(self.logits, self.targets, self.stats, self.entropy, self.d_logprob,
                                       self.d_entropy, 1.0)
        dy = dlogits @ self.table
        dtable = dlogits.t() @ self.y                             # the output layer's share, bf16
        dx, dw = nf.fused_add_rmsnorm_bwd(dy, self.res, self.w, None, EPS)
        dx0 = (dx.float() + (dx @ self.branch.t()).float()).bfloat16()
        nf.embedding_bwd(dx0, self.ids, self.vocab, self.scale, accumulate=dtable)
        return dtable, dw


def exact(m, table, w):
    """logprob and entropy of the model in 64 bits."""
    keep = (m.ids >= 0).double()[:, None]
    x0 = table[m.ids.clamp(min=0)] * m.scale * keep
    s = x0 + x0 @ m.branch.double()
    y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * w
    log_p = torch.log_softmax(y @ table.t(), 1)
    entropy = -(log_p.exp() * log_p).sum(1)
    logprob = log_p.gather(1, m.targets.clamp(min=0)[:, None])[:, 0] * (m.targets >= 0)
    return logprob, entropy


def test_training_step():
    m = Model()
    logprob, entropy = m.forward()
    table, w = m.table.double().requires_grad_(), m.w.double().requires_grad_()
    ref_lp, ref_ent = exact(m, table, w)
    dtable, dw = m.backward()
    loss = (m.d_logprob.double() * ref_lp + m.d_entropy.double() * ref_ent).sum()
    ref_dtable, ref_dw = torch.autograd.grad(loss, (table, w))

    def off(got, ref):
        return ((got.double() - ref).norm() / ref.norm()).item()
    # forward: x0, branch output, stream, y and logits are rounded; backward: dlogits, dy, dx, branch, dx0, dtable too
    assert off(logprob, ref_lp.detach()) < 4 * 5 * 2.0 ** -8
    assert off(entropy, ref_ent.detach()) < 4 * 5 * 2.0 ** -8
    assert off(dtable, ref_dtable) < 4 * 11 * 2.0 ** -8
    assert off(dw, ref_dw) < 4 * 8 * 2.0 ** -8
    # the alternatives are the logits' own
    best, ids = torch.sort(m.logits.double(), dim=1, descending=True, stable=True)
    assert torch.equal(m.top_ids, ids[:, :4])
    assert torch.all(m.top[:, 0] >= m.top[:, 1])


def test_training_step_is_reproducible_and_captures():
    m = Model(seed=1)
    m.forward()
    want = m.backward()
    again = m.backward()
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the libraries' own first calls, before the capture
        m.forward()
        m.backward()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp, ent = m.forward()
        got = m.backward()
    for _ in range(3):
        for t in (lp, ent) + got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_serving_step_with_8_bit_rows():
    m = Model(tokens=96, hidden=1024, seed=2)
    x0 = nf.embedding_fwd(m.ids, m.table, m.scale)
    y = x0 @ m.branch
    ref_res, ref_y = x0.clone(), y.clone()
    nf.fused_add_rmsnorm(ref_y, ref_res, m.w, EPS)
    for fmt, step in (("e4m3", 2.0 ** -4), ("int8", 0.5 / 127)):
        for group in (0, 128):
            res = x0.clone()
            q, scale = nf.fused_add_rmsnorm_q8(y, res, m.w, EPS, fmt=fmt, group=group)
            assert torch.equal(res, ref_res)
            s = scale.repeat_interleave(128, 1) if group else scale[:, None]
            rows = q.float() * s
            # against the bf16 operator: half a step of the 8-bit value (of the largest one, for int8) and
            # half a bf16 step; below e4m3's normal numbers the step is 2^-9 of the scale
            largest = ref_y.float().abs().amax(1, keepdim=True)
            tol = (ref_y.float().abs() * step + s * 2.0 ** -10 if fmt == "e4m3" else largest * step) * 1.01 + 2.0 ** -7 * ref_y.float().abs()
            assert torch.all((rows - ref_y.float()).abs() <= tol + 1e-6)
            logits = rows.bfloat16() @ m.table.t()
            lp, ent, _, top, ids = nf.token_logprob_fwd(logits, m.targets, 0.7, top=1)
            given = m.targets >= 0
            assert torch.isfinite(lp).all() and torch.all(lp[~given] == 0)
            assert torch.all(top[:, 0][given] >= lp[given] - 1e-5)
            nxt = nf.embedding_fwd(ids[:, 0], m.table, m.scale)   # the next step's rows
            assert torch.equal(nxt, nf.embedding_fwd(ids[:, 0].int(), m.table, m.scale))


FRESH = r"""
import torch
import row_normalization_inner_gb300 as nf
g = torch.Generator(device="cuda")
g.manual_seed(1)
# the entry points' first calls, at their smallest
x = torch.randn(2, 64, generator=g, device="cuda").bfloat16()
w = torch.ones(64, device="cuda").bfloat16()
nf.rmsnorm_q8(x, w)
nf.fused_add_rmsnorm_q8(x, x.clone(), w)
ids = torch.tensor([1, 0], device="cuda")
nf.embedding_fwd(ids, x)
nf.embedding_bwd(x, ids, 5)
lp, ent, stats, _, _ = nf.token_logprob_fwd(x, ids)
nf.token_logprob_bwd(x, ids, stats, ent, lp)
torch.cuda.synchronize()
# other kernels of the same entry points, met for the first time inside a capture
x = torch.randn(2500, 4104, generator=g, device="cuda").bfloat16()
r = torch.randn(2500, 4104, generator=g, device="cuda").bfloat16()
w = torch.randn(4104, generator=g, device="cuda").bfloat16()
ids = torch.randint(-1, 3000, (2500,), generator=g, device="cuda")
many = torch.randint(-1, 3000, (40000,), generator=g, device="cuda")
some = torch.randint(-1, 3000, (20000,), generator=g, device="cuda")
dy = torch.randn(40000, 64, generator=g, device="cuda").bfloat16()
table = torch.randn(3000, 4104, generator=g, device="cuda").bfloat16()
logits = torch.randn(20, 40001, generator=g, device="cuda")
t = torch.randint(0, 40001, (20,), generator=g, device="cuda").int()

def step():
    res = r.clone()
    out = list(nf.rmsnorm_q8(x, w, fmt="int8")) + list(nf.rmsnorm_q8(x, w, group=128))
    out += list(nf.fused_add_rmsnorm_q8(x, res, w, group=128)) + [res]
    out += [nf.embedding_fwd(ids, table, 3.0), nf.embedding_bwd(x, ids, 3000, dtype=torch.bfloat16)]
    out += [nf.embedding_bwd(dy, many, 3000), nf.embedding_bwd(dy[:20000], some, 3000)]
    lp, ent, stats, top, top_ids = nf.token_logprob_fwd(logits, t, 0.5, top=32)
    return out + [lp, ent, stats, top, top_ids, nf.token_logprob_bwd(logits, t, stats, ent, lp, ent, 0.5)]

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
assert nf.nf_get_device_status(0) == nf.NF_OK
print("captured")
"""


def test_kernels_first_met_inside_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FRESH], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_calls_at_once_on_two_streams():
    m = Model(tokens=3000, vocab=5003, hidden=1024, seed=3)
    dy = torch.randn(3000, 1024, device="cuda").bfloat16()
    logits = torch.randn(3000, 5003, device="cuda")

    def step(ids, targets):
        y = nf.embedding_fwd(ids, m.table, 2.0)
        q, scale = nf.rmsnorm_q8(y, m.w, EPS)
        lp, ent, stats, top, top_ids = nf.token_logprob_fwd(logits, targets, top=8)
        return [y, q, scale, lp, ent, top, top_ids, nf.embedding_bwd(dy, ids, 5003),
                nf.token_logprob_bwd(logits, targets, stats, ent, m.d_logprob)]
    inputs = [(m.ids, m.targets), (m.ids.flip(0), m.targets.flip(0))]
    want = [step(*i) for i in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    for _ in range(5):
        got = []
        for s, i in zip(streams, inputs):
            with torch.cuda.stream(s):
                got.append(step(*i))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_calls_from_several_threads():
    # the helpers let the interpreter go while they allocate and launch
    from concurrent.futures import ThreadPoolExecutor
    vocab, hidden, tokens, rows = 3000, 256, 900, 7

    def inputs(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        ids = torch.randint(-1, vocab, (tokens,), generator=g, device="cuda")
        return r(tokens, hidden).bfloat16(), ids, r(rows, vocab).bfloat16(), ids[:rows].contiguous(), r(hidden).bfloat16()

    def calls(dy, ids, logits, targets, w):
        return [nf.embedding_bwd(dy, ids, vocab), *nf.rmsnorm_q8(dy, w, group=128),
                *nf.token_logprob_fwd(logits, targets, top=4)]

    given = [inputs(s) for s in range(4)]
    want = [calls(*x) for x in given]
    torch.cuda.synchronize()

    def work(x):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = calls(*x)
            torch.cuda.current_stream().synchronize()
        return got

    with ThreadPoolExecutor(4) as pool:
        for got, ref in zip(pool.map(work, given), want):
            for a, b in zip(got, ref):
                assert torch.equal(a.view(torch.uint8) if a.dtype == torch.float8_e4m3fn else a,
                                   b.view(torch.uint8) if b.dtype == torch.float8_e4m3fn else b)
