"""Rows of heads that lie far apart, rows between one another's, and the sums of
the weights' gradients over many rows of few heads.

A row's bits do not depend on where it lies, so far rows are compared with the
same rows side by side, for equality.

The sums.  A lane adds one product a pass to its columns' sums.  With T tokens
whose heads take p_i passes each (32 / G heads to a pass, G lanes to a row; one
head in the element kernel), P = sum T p_i passes of all kinds take min(3 SMs,
P / 8) CTAs of four warps, shared out by p_i (+ 1 for a token's angles in the
vector kernel): kind i has ctas_i CTAs and chains of T p_i / (4 ctas_i) + 1
additions.  Behind a chain come at most 31 over the warp's groups, 3 over the
CTA's warps, 2 over every 256th CTA and 12 over these: depth + 48 roundings of u =
2^-24 of the sum of the terms' magnitudes, beside what the terms are off.
"""
import pytest
import torch

import row_normalization_inner_gb300 as nf
from heads_reference import close, frequencies, gen, heads, norm_turn_grad, normed, rates_of, turn

pytestmark = pytest.mark.gpu

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    yield


FAR = 2 ** 30 + 64  # elements: the third row is beyond 2^31
ORDERS = {"tokens": (3 * FAR + 128, FAR, None), "heads": (None, None, FAR), "batches": (2 ** 31 + 192, None, None)}


def far(x, order):
    """A copy of x [batch, tokens, heads, dim] whose rows lie far apart; all else of its memory is left as it comes."""
    b, t, h, d = x.shape
    close_by = (t * h * d, h * d, d)
    strides = [s or c for s, c in zip(ORDERS[order], close_by)]
    room = sum((n - 1) * s for n, s in zip((b, t, h), strides)) + d
    y = torch.empty(room, dtype=x.dtype, device="cuda").as_strided(x.shape, (*strides, 1))
    return y.copy_(x)


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("kind,dim", [(BF, 64), (BF, 20), (F32, 80)])  # (20: element by element)
def test_far_rows(kind, dim, order):
    g = gen(41)
    x, dy, w = heads(g, 2, 3, 3, dim, kind=kind), heads(g, 2, 3, 3, dim, kind=kind), heads(g, dim, kind=kind)
    rot = dim // 2 // 16 * 16 or dim // 2
    rates = rates_of(rot)
    positions = torch.randint(0, 5000, (2, 3), generator=g, device="cuda")
    want = nf.rope_fwd(x, None, positions, rates)[0], nf.qk_rmsnorm_rope_fwd(x, None, w, None, positions, rates)[0]
    back = nf.qk_rmsnorm_rope_bwd(dy, None, x, None, w, None, positions, rates)
    a, out = far(x, order), far(torch.zeros_like(x), order)
    assert torch.equal(nf.rope_fwd(a, None, positions, rates, q_out=out)[0], want[0])
    assert torch.equal(nf.qk_rmsnorm_rope_fwd(a, None, w, None, positions, rates, q_out=out)[0], want[1])
    got = nf.qk_rmsnorm_rope_bwd(far(dy, order), None, a, None, w, None, positions, rates, dq=out)
    assert got[0] is out and torch.equal(out, back[0]) and torch.equal(got[2], back[2])
    # in the input's own place
    assert torch.equal(nf.qk_rmsnorm_rope_bwd(dy, None, a, None, w, None, positions, rates, dq=a)[0], back[0])
    # and of an append
    k, v = far(x, order)[0], far(dy, order)[0]
    caches, near = [torch.zeros(2, 4, 1, 3, dim, dtype=kind, device="cuda") for _ in range(2)]
    table, past = torch.tensor([[2], [0], [3]], dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    q = nf.kv_append(k, v, caches[0], caches[1], table, past, rates=rates, positions=positions[0], q=k, q_out=out[0])
    assert torch.equal(q, want[0][0])
    nf.kv_append(x[0], dy[0], near[0], near[1], table, past, rates=rates, positions=positions[0])
    assert torch.equal(caches, near) and torch.equal(caches[1][[2, 0, 3], 0], dy[0])


def test_far_positions_of_a_batch():
    g = gen(42)
    q, rates = heads(g, 2, 3, 2, 64), rates_of(64)
    near = torch.randint(0, 5000, (2, 3), generator=g, device="cuda", dtype=torch.int32)
    positions = torch.empty(2 ** 31 + 8, dtype=torch.int32, device="cuda").as_strided((2, 3), (2 ** 31 + 5, 1)).copy_(near)
    assert torch.equal(nf.rope_fwd(q, None, positions, rates)[0], nf.rope_fwd(q, None, near, rates)[0])


@pytest.mark.parametrize("dim", [128, 20])
def test_heads_in_turn_under_a_padded_token(dim):
    # a query, a key and a value in turn, tokens 16 elements further apart than the heads fill: in place, and back
    g = gen(43)
    tokens, n = 50, 4
    room = torch.randn(tokens, n * 3 * dim + 16, generator=g, device="cuda").bfloat16()
    keep = room.clone()
    q, k, v = room[:, :n * 3 * dim].view(tokens, n, 3, dim).unbind(2)
    p, rates, w = torch.arange(tokens, device="cuda"), rates_of(dim), heads(g, dim)
    want = nf.qk_rmsnorm_rope_fwd(q, k, w, w, p, rates)
    back = nf.qk_rmsnorm_rope_bwd(want[0], want[1], q, k, w, w, p, rates)
    got = nf.qk_rmsnorm_rope_fwd(q, k, w, w, p, rates, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(room[:, n * 3 * dim:], keep[:, n * 3 * dim:]) and torch.equal(v, keep[:, :n * 3 * dim].view(tokens, n, 3, dim)[:, :, 2])
    room.copy_(keep)
    got = nf.qk_rmsnorm_rope_bwd(want[0], want[1], q, k, w, w, p, rates, dq=q, dk=k)
    assert all(torch.equal(a, b) for a, b in zip((q, k, got[2], got[3]), back))


@pytest.mark.parametrize("cell", [BF, E4M3])
def test_a_cache_of_a_heads_keys_beside_its_values(cell):
    # pages of [heads, 2, page_size, dim]
    g = gen(44)
    tokens, pages, page, n, dim = 70, 9, 8, 3, 64
    k, v = heads(g, tokens, n, dim), heads(g, tokens, n, dim)
    table = torch.arange(8, -1, -1, dtype=torch.int32, device="cuda")[None]
    past, starts = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, tokens], dtype=torch.int32, device="cuda")

    def run(cache, scale):
        kw = dict(k_scale=scale[0], v_scale=scale[1]) if cell != BF else {}
        nf.kv_append(k, v, cache[0], cache[1], table, past, starts, rates_of(dim), **kw)
        return [t.float() for t in cache] + list(scale)
    both, scales = torch.zeros(pages, n, 2, page, dim, device="cuda").to(cell), torch.zeros(pages, n, 2, page, device="cuda")
    got = run([both[:, :, i].transpose(1, 2) for i in range(2)], [scales[:, :, i].transpose(1, 2) for i in range(2)])
    want = run([torch.zeros(pages, page, n, dim, device="cuda").to(cell) for _ in range(2)], [torch.zeros(pages, page, n, device="cuda") for _ in range(2)])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and want[0].any()


def depth(tokens, counts, kind, dim, vectors):
    """The longest chain of additions of each kind of heads."""
    W = 8 if kind == BF else 4
    lanes = dim // (2 * W) if vectors else 32
    passes = [tokens * -(-n // (32 // lanes)) for n in counts]
    work = [p + (tokens if vectors else 0) for p in passes]
    ctas = max(len(counts), min(3 * torch.cuda.get_device_properties(0).multi_processor_count, sum(passes) // 8))
    return [p // (4 * max(1, int(ctas * w / sum(work)) - 1)) + 1 for p, w in zip(passes, work)]


@pytest.mark.parametrize("kind,dim,hq,hk,tokens", [(BF, 128, 64, 1, 16384), (BF, 64, 3, 1, 30001), (F32, 128, 16, 2, 9000), (BF, 20, 40, 1, 5000), (F32, 7, 12, 3, 3000)])
def test_sums_over_many_rows_of_few_heads(kind, dim, hq, hk, tokens):
    g = gen(45)
    q, k, dq, dk = [heads(g, tokens, n, dim, kind=kind) for n in (hq, hk, hq, hk)]
    qw, kw = heads(g, dim, kind=kind), heads(g, dim, kind=kind)
    rot, p = dim // 2 * 2, torch.arange(tokens, device="cuda")
    got = nf.qk_rmsnorm_rope_bwd(dq, dk, q, k, qw, kw, p, rates_of(rot), EPS)
    for dx, dw, dy, x, w, chain in zip(got[:2], got[2:], (dq, dk), (q, k), (qw, kw), depth(tokens, (hq, hk), kind, dim, dim >= 64)):
        rdx, rdw, off, _ = norm_turn_grad(dy, x, w, EPS, p, frequencies(rot))
        close(dx, rdx, off)
        _, size = turn(dy, p, frequencies(rot), back=True)
        terms = (size * normed(x, torch.ones_like(w), EPS).abs()).flatten(0, -2).sum(0)
        close(dw, rdw, terms * (2.0 ** -17 + (chain + 48) * 2.0 ** -24))
