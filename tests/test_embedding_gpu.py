"""Embedding lookup and its gradient against the definition in 64 bits.

Tolerances.  The lookup rounds scale * table once to fp32 (2^-24 relative)
and once to bf16 (2^-8).  A gradient entry sums m values in fp32 in some
order, each addition off by at most 2^-24 of a partial sum, so by at most
m * 2^-24 * sum |dy|; the scaling and the addition of the old value round
once each, and a bf16 result once more.
"""
import math

import pytest
import torch

import row_normalization_inner_gb300 as nf

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    yield


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make_ids(kind, n, vocab, seed):
    g = gen(seed)
    if kind == "uniform":
        ids = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    elif kind == "words":  # density 1 / id, some outside the table
        u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * math.log(vocab + 1.0)).long() - 1).clamp(0, vocab - 1)
        ids[::7] = -1
        ids[3::11] = vocab
        ids[5::13] = -100
    elif kind == "one":
        ids = torch.full((n,), vocab - 1, device="cuda")
    elif kind == "none":
        ids = torch.full((n,), -1, device="cuda")
    elif kind == "falling":
        ids = (torch.arange(n, 0, -1, device="cuda") - 1) * vocab // max(n, 1)
    else:
        raise ValueError(kind)
    return ids.long()


# ---------------------------------------------------------------- lookup

@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("tokens,vocab,hidden", [(1, 1, 8), (5, 7, 64), (33, 1000, 1000), (300, 50, 4096),
                                                 (1000, 32003, 264), (17, 11, 12288), (2, 3, 40008)])
def test_lookup(tokens, vocab, hidden, wide):
    ids = make_ids("words", tokens, vocab, tokens)
    table = torch.randn(vocab, hidden, generator=gen(1), device="cuda").bfloat16()
    if not wide:
        ids = ids.int()
    for scale in (1.0, math.sqrt(hidden), -0.37):
        y = nf.embedding_fwd(ids, table, scale)
        known = (ids >= 0) & (ids < vocab)
        ref = table.double()[ids.long().clamp(0, vocab - 1)] * scale * known[:, None]
        assert torch.all((y.double() - ref).abs() <= (HALF + 2 * U) * ref.abs())
        if scale == 1.0:
            assert torch.equal(y.double(), ref)


def test_lookup_far_rows_shapes_and_outputs():
    # row offsets beyond 2^31 elements
    table = torch.zeros(1 << 19, 4104, dtype=torch.bfloat16, device="cuda")
    assert table.numel() > 1 << 31
    table[-1] = 3.0
    table[-2] = 2.0
    ids = torch.tensor([[(1 << 19) - 1, -1], [(1 << 19) - 2, 1 << 19], [(1 << 40) + 1, 0]], device="cuda")
    y = nf.embedding_fwd(ids, table)
    assert y.shape == (3, 2, 4104)
    assert torch.all(y[0, 0] == 3) and torch.all(y[1, 0] == 2) and torch.all(y[:, 1] == 0) and torch.all(y[2, 0] == 0)
    out = torch.empty_like(y)
    assert nf.embedding_fwd(ids, table, out=out) is out and torch.equal(out, y)
    assert nf.embedding_fwd(ids[:0], table).shape == (0, 2, 4104)
    with pytest.raises(ValueError):
        nf.embedding_fwd(ids, table, out=out[:, :1])
    with pytest.raises(ValueError):
        nf.embedding_fwd(ids.t(), table)
    with pytest.raises(ValueError):
        nf.embedding_fwd(ids, table[0])
    with pytest.raises(nf.NFError):
        nf.embedding_fwd(ids, table, float("inf"))


# ---------------------------------------------------------------- gradient

def check_grad(got, dy, ids, vocab, scale, old, rows=None):
    keep = (ids >= 0) & (ids < vocab)
    at = ids.long()[keep].flatten()
    d = dy.double()[keep].view(-1, dy.shape[-1]) * scale
    hidden = dy.shape[-1]
    ref = torch.zeros(vocab, hidden, dtype=torch.float64, device="cuda").index_add_(0, at, d)
    size = torch.zeros_like(ref).index_add_(0, at, d.abs())
    m = torch.zeros(vocab, dtype=torch.float64, device="cuda").index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    tol = (m[:, None] + 2) * U * size
    if old is not None:
        ref = ref + old.double()
        tol = tol + 2 * U * ref.abs()
    if got.dtype == torch.bfloat16:
        tol = tol + HALF * (ref.abs() + tol)
    assert torch.all((got.double() - ref).abs() <= tol)
    untouched = m == 0
    if old is None:
        assert torch.all(got[untouched] == 0)
    else:
        assert torch.equal(got[untouched], old[untouched])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("kind", ["uniform", "words", "one", "none", "falling"])
@pytest.mark.parametrize("tokens,vocab,hidden", [
    (1, 1, 8), (1, 1000, 64), (9, 3, 1000), (257, 1023, 128), (1000, 1024, 136), (4097, 131072, 64),
    (16384, 5000, 1032), (16385, 300, 40), (20011, 70000, 256), (70001, 32003, 264), (5000, 1 << 21, 16),
    (40000, 1 << 21, 16)])
def test_gradient(tokens, vocab, hidden, kind, add, dtype):
    ids = make_ids(kind, tokens, vocab, tokens + vocab)
    g = gen(tokens)
    dy = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    old = torch.randn(vocab, hidden, generator=g, device="cuda").to(dtype)
    if add:
        got = old.clone()
        assert nf.embedding_bwd(dy, ids, vocab, 0.5, accumulate=got) is got
        check_grad(got, dy, ids, vocab, 0.5, old)
    else:
        out = torch.full((vocab, hidden), float("nan"), dtype=dtype, device="cuda")
        got = nf.embedding_bwd(dy, ids, vocab, 0.5, out=out)
        assert got is out
        check_grad(got, dy, ids, vocab, 0.5, None)


@pytest.mark.parametrize("kind", ["words", "one", "falling"])
@pytest.mark.parametrize("tokens", [31, 32, 33, 4095, 4096, 8193, 16384, 16390, 32768, 32769, 65537])
def test_gradient_at_the_borders_of_the_sorts(tokens, kind):
    vocab, hidden = 3001, 16
    ids = make_ids(kind, tokens, vocab, tokens)
    dy = torch.randn(tokens, hidden, generator=gen(tokens), device="cuda").bfloat16()
    check_grad(nf.embedding_bwd(dy, ids, vocab, 1.0), dy, ids, vocab, 1.0, None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,vocab,hidden", [(40, 5000, 8), (600, 5001, 24), (40, 2049, 96), (600, 130, 4104),
                                                 (40, 7, 32768), (600, 1025, 16), (5, 1 << 20, 8)])
def test_zeros_of_rows_without_tokens(tokens, vocab, hidden, dtype):
    # rows of many lengths, many or one to a CTA; every element of the table was something else before
    ids = make_ids("words", tokens, vocab, tokens)
    dy = torch.randn(tokens, hidden, generator=gen(tokens), device="cuda").bfloat16()
    out = torch.full((vocab, hidden), float("nan"), dtype=dtype, device="cuda")
    check_grad(nf.embedding_bwd(dy, ids, vocab, dtype=dtype, out=out), dy, ids, vocab, 1.0, None)


@pytest.mark.parametrize("dtype,add", [(torch.float32, False), (torch.bfloat16, True)])
@pytest.mark.parametrize("kind", ["uniform", "words", "one", "falling"])
@pytest.mark.parametrize("tokens,vocab,hidden", [
    (2, 1, 512), (8, 3, 520), (9, 40, 4104), (17, 2, 1032), (127, 8, 8), (255, 30, 16392), (256, 2000, 248),
    (511, 60, 1000), (512, 32003, 2056), (512, 3, 504), (513, 60, 1000)])
def test_gradient_of_few_tokens(tokens, vocab, hidden, kind, dtype, add):
    # one launch up to 512 tokens; runs of a warp (8 rows) and of the whole CTA
    ids = make_ids(kind, tokens, vocab, tokens + hidden)
    g = gen(tokens)
    dy = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    old = torch.randn(vocab, hidden, generator=g, device="cuda").to(dtype) if add else None
    got = nf.embedding_bwd(dy, ids, vocab, 1.7, dtype=dtype, accumulate=None if old is None else old.clone())
    check_grad(got, dy, ids, vocab, 1.7, old)
    again = nf.embedding_bwd(dy, ids, vocab, 1.7, dtype=dtype, accumulate=None if old is None else old.clone())
    assert torch.equal(got, again)


@pytest.mark.parametrize("kind", ["uniform", "words", "one", "none"])
@pytest.mark.parametrize("tokens,vocab", [(98305, 5), (131072, 70000), (131073, 1 << 21), (400001, 40000)])
def test_gradient_of_many_tiles(tokens, vocab, kind):
    # counts of the digits summed over the tiles by a launch of their own
    hidden = 8
    ids = make_ids(kind, tokens, vocab, tokens)
    dy = torch.randn(tokens, hidden, generator=gen(tokens), device="cuda").bfloat16()
    check_grad(nf.embedding_bwd(dy, ids, vocab, 0.5), dy, ids, vocab, 0.5, None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hidden", [8, 64, 264])
@pytest.mark.parametrize("tokens,vocab", [(70001, 1500), (200000, 131072), (200000, 1), (1 << 20, 5003)])
def test_zeros_beside_frequent_ids(tokens, vocab, hidden, dtype):
    # the rows that one CTA writes hold a large part of all tokens, or all of them, every third row none
    ids = make_ids("words", tokens, vocab, 7)
    ids = torch.where(ids % 3 == 1, 0, ids)
    dy = torch.randn(tokens, hidden, generator=gen(8), device="cuda").bfloat16()
    out = torch.full((vocab, hidden), float("nan"), dtype=dtype, device="cuda")
    check_grad(nf.embedding_bwd(dy, ids, vocab, dtype=dtype, out=out), dy, ids, vocab, 1.0, None)


def test_frequent_ids_do_not_hold_up_the_zeros():
    # the CTA that writes the zeros around the most frequent ids must not take
    # a time of its own that grows with the tokens: written and added differ by
    # the zeros, which take 2 us here (4 MB), and not by the ids' distribution
    tokens, vocab, hidden = 1 << 22, 131072, 8
    dy = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    ids = torch.randint(0, 100, (tokens,), generator=gen(9), device="cuda")
    out = torch.zeros(vocab, hidden, device="cuda")
    ws = torch.empty(nf.nf_embedding_bwd_workspace_size(tokens, hidden), dtype=torch.uint8, device="cuda")

    def time(**kw):
        best = math.inf
        for _ in range(5):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            nf.embedding_bwd(dy, ids, vocab, workspace=ws, **kw)
            end.record()
            end.synchronize()
            best = min(best, start.elapsed_time(end))
        return best
    # 1.0 measured, and 2.2 where that CTA walks all the tokens
    assert time(out=out) < 1.5 * time(accumulate=out)


@pytest.mark.parametrize("tokens", [3000, 30000])
def test_gradient_is_deterministic_and_in_token_order(tokens):
    vocab, hidden = 500, 520
    ids = make_ids("words", tokens, vocab, 3)
    dy = torch.randn(tokens, hidden, generator=gen(4), device="cuda").bfloat16()
    first = nf.embedding_bwd(dy, ids, vocab, 2.0)
    for _ in range(3):
        assert torch.equal(nf.embedding_bwd(dy, ids, vocab, 2.0), first)
    assert torch.equal(nf.embedding_bwd(dy, ids.int(), vocab, 2.0), first)
    # each run is the ordered sum of its rows, so moving other ids' tokens changes nothing but chunk borders:
    # a batch of one id per row is exact
    ids = torch.randperm(vocab, generator=gen(5), device="cuda")
    dy = torch.randn(vocab, hidden, generator=gen(6), device="cuda").bfloat16()
    got = nf.embedding_bwd(dy, ids, vocab, 1.0)
    assert torch.equal(got[ids], dy.float())


@pytest.mark.parametrize("runs", [60, 500, 2500, 10000])
def test_runs_within_a_piece_are_summed_in_token_order(runs):
    # every id eight times: a run of one warp (480 tokens), or inside one chunk, whose lengths are powers of two
    # from 8 on.  Magnitudes from 2^-12 to 2^12 round differently in another order.
    each, hidden = 8, 72
    tokens = runs * each
    ids = torch.arange(runs, device="cuda").repeat(each)[torch.randperm(tokens, generator=gen(1), device="cuda")]
    dy = torch.randn(tokens, hidden, generator=gen(2), device="cuda")
    dy = (dy * torch.exp2(torch.randint(-12, 13, dy.shape, generator=gen(3), device="cuda").float())).bfloat16()
    rows = dy[torch.sort(ids, stable=True).indices].float().view(runs, each, hidden)

    def in_order(which):
        total = torch.zeros(runs, hidden, device="cuda")
        for k in which:
            total = total + rows[:, k]
        return total
    want = in_order(range(each))
    assert not torch.equal(in_order(reversed(range(each))), want)
    assert torch.equal(nf.embedding_bwd(dy, ids, runs), want)
    assert torch.equal(nf.embedding_bwd(dy, ids, runs, accumulate=torch.zeros(runs, hidden, device="cuda")), want)
    assert torch.equal(nf.embedding_bwd(dy, ids, runs, dtype=torch.bfloat16), want.bfloat16())


def test_gradient_far_rows():
    vocab, hidden = (1 << 19) + 3, 4104  # offsets beyond 2^31 elements
    ids = torch.tensor([vocab - 1, 5, vocab - 1, vocab], device="cuda")
    dy = torch.ones(4, hidden, device="cuda").bfloat16()
    got = nf.embedding_bwd(dy, ids, vocab, 1.0, dtype=torch.bfloat16)
    assert torch.all(got[vocab - 1] == 2) and torch.all(got[5] == 1)
    assert int((got != 0).any(1).sum()) == 2
    nf.embedding_bwd(dy, ids, vocab, 1.0, accumulate=got)
    assert torch.all(got[vocab - 1] == 4) and torch.all(got[5] == 2)


def test_gradient_empty_batch_and_refusals():
    dy = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    out = torch.full((100, 64), 7.0, device="cuda")
    assert torch.all(nf.embedding_bwd(dy, ids, 100, accumulate=out) == 7)
    assert torch.all(nf.embedding_bwd(dy, ids, 100, out=out) == 0)
    dy = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        nf.embedding_bwd(dy, ids[:3], 100)
    with pytest.raises(ValueError):
        nf.embedding_bwd(dy, ids, 99, out=out)
    with pytest.raises(ValueError):
        nf.embedding_bwd(dy, ids, 100, out=out, accumulate=out)
    with pytest.raises(TypeError):
        nf.embedding_bwd(dy, ids, 100, dtype=torch.float16)
    with pytest.raises(TypeError):
        nf.embedding_bwd(dy, ids, 100, dtype=torch.bfloat16, out=out)
    with pytest.raises(ValueError):
        nf.embedding_bwd(dy.t(), ids.expand(64, 4), 100)
    with pytest.raises(nf.NFError):
        nf.embedding_bwd(dy, ids, 100, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("tokens", [700, 20000])
def test_another_stream_and_graphs_that_share_a_workspace(tokens):
    vocab, hidden = 3000, 256
    dy = torch.randn(tokens, hidden, generator=gen(1), device="cuda").bfloat16()
    ids = [make_ids("words", tokens, vocab, s) for s in (1, 2)]
    want = [nf.embedding_bwd(dy, i, vocab) for i in ids]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = nf.embedding_bwd(dy, ids[0], vocab, stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
    ws = torch.empty(nf.nf_embedding_bwd_workspace_size(tokens, hidden), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for i in ids:
        out = torch.zeros(vocab, hidden, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            nf.embedding_bwd(dy, i, vocab, out=out, workspace=ws)
        graphs.append(g)
        outs.append(out)
    for k in (0, 1, 1, 0, 1):
        outs[k].fill_(float("nan"))
        graphs[k].replay()
        assert torch.equal(outs[k], want[k])
