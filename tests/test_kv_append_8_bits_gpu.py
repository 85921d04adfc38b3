"""Rows of an 8-bit cache to the last bit.

Values go to the cache as they are, so their 8-bit rows have one right result:
scale = max(max|v| / Q, 2^-100) and q = v / scale, each quotient rounded to fp32
once, and q then to the nearest value of its format, ties to even.  The scale and
the rows are compared with that, computed in numpy: for equality, no tolerance.
Rows of 16-bit values have quotients exactly between two 8-bit values all the
time (every 16th of a row whose maximum is 7 * 2^k), and it is these that a
quotient without its last bit, or another way with ties, gets wrong.

Keys are turned before they are rounded, with the bounds of heads_reference: q
is within half a step of its own binade (2^(floor(log2 |y / scale|) - 4) in e4m3),
not of the largest that its magnitude could have.
"""
import numpy as np
import pytest
import torch

import row_normalization_inner_gb300 as nf
from heads_reference import TURN, frequencies, gen, turn

pytestmark = pytest.mark.gpu

BF, F32, E4M3, INT8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8
QMAX = {E4M3: np.float32(448), INT8: np.float32(127)}
PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    yield


def nearest(v, cell):
    """fp32 numbers to the nearest of the format, ties to even; and which of them are ties."""
    v = v.astype(np.float64)
    if cell == INT8:
        step = np.ones_like(v)
    else:  # 3 mantissa bits, smallest normal exponent -6: |v| = m * 2^e with m in [1/2, 1)
        step = np.exp2(np.maximum(np.frexp(v)[1] - 1, -6) - 3.0)
    t = v / step  # exact: the steps are powers of two
    return np.clip(np.rint(t) * step, -float(QMAX[cell]), float(QMAX[cell])), np.abs(t - np.floor(t)) == 0.5


def rows_8(v, cell):
    """(q, scale, ties) of rows [..., dim] in fp32."""
    scale = np.maximum(np.abs(v).max(-1) / QMAX[cell], np.float32(2.0 ** -100))
    assert scale.dtype == np.float32
    q, ties = nearest(v / scale[..., None], cell)
    return q, scale, ties


def values(g, tokens, heads, dim, kind, cell):
    """Normal rows of many sizes; every other one with a maximum whose scale is a power of two and elements of few bits, a quarter of them ties."""
    v = torch.randn(tokens, heads, dim, generator=g, device="cuda") * torch.exp2(torch.randint(-20, 20, (tokens, heads, 1), generator=g, device="cuda"))
    power = torch.exp2(torch.randint(-12, 12, (tokens, heads, 1), generator=g, device="cuda").float())
    most, steps = (7.0, 2.0 ** -3) if cell == E4M3 else (127.0, 0.5)
    even = torch.randint(-int(most / steps) + 1, int(most / steps), v.shape, generator=g, device="cuda") * steps * power
    at = torch.randint(0, dim, (tokens, heads, 1), generator=g, device="cuda")
    even.scatter_(2, at, most * power * torch.where(at % 2 == 0, 1.0, -1.0))
    return torch.where(((torch.arange(tokens * heads, device="cuda") % 2) == 0).view(tokens, heads, 1), v, even).to(kind)


# few rows, and enough that a warp takes several, of one token and of many; keys and values apart and in one share; heads whose lanes all
# have two vectors, others, and heads that go element by element
SHAPES = [(3, 4, 1, 64), (5, 8, 2, 128), (2, 3, 3, 80), (7, 2, 1, 72), (4, 2, 2, 20), (6, 1, 1, 7), (2, 2, 1, 256), (3, 1, 2, 192), (3, 1, 1, 512),
          (1700, 64, 8, 128), (1500, 32, 8, 128), (1501, 32, 4, 80), (4003, 8, 1, 128), (3001, 5, 1, 64), (1300, 6, 6, 72), (1200, 17, 9, 64), (900, 4, 4, 20)]


@pytest.mark.parametrize("cell", [E4M3, INT8])
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("tokens,hq,hk,dim", SHAPES)
def test_values_to_the_last_bit(tokens, hq, hk, dim, kind, cell):
    g = gen(tokens + hk + dim)
    pages = -(-tokens // PAGE)
    k, v = values(g, tokens, hk, dim, kind, cell), values(g, tokens, hk, dim, kind, cell)
    q = torch.randn(tokens, hq, dim, generator=g, device="cuda").to(kind)
    table = torch.randperm(pages, generator=g, device="cuda").int()[None]
    past, starts = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    place = torch.arange(tokens, device="cuda")
    at = (table[0].long()[place // PAGE], place % PAGE)

    def appended(**kw):
        caches = [torch.zeros(pages, PAGE, hk, dim, dtype=cell, device="cuda") for _ in range(2)]
        scales = [torch.zeros(pages, PAGE, hk, device="cuda") for _ in range(2)]
        nf.kv_append(k, v, *caches, table, past, starts, k_scale=scales[0], v_scale=scales[1], **kw)
        return [(c[at].float().cpu().numpy(), s[at].cpu().numpy()) for c, s in zip(caches, scales)]

    def same(got, x, ties_too):
        want, scale, ties = rows_8(x.float().cpu().numpy(), cell)
        # a third of the rows or more are made for it, a quarter of their elements ties
        assert not ties_too or dim < 64 or ties.mean() > 1 / 40
        assert np.array_equal(got[1], scale), np.abs(got[1] / scale - 1).max()
        bad = got[0] != want
        assert not bad.any(), (int(bad.sum()), bad.size, got[0][bad][:4], want[bad][:4], ties[bad][:4])

    plain = appended()  # keys neither normalized nor turned are such rows too
    same(plain[0], k, True)
    same(plain[1], v, True)
    rot = dim // 2 * 2
    for layout in ("half", "interleaved"):
        turned = appended(q=q, rates=nf.rope_rates(rot), layout=layout, k_weight=None)
        same(turned[1], v, True)
        y, size = turn(k, place, frequencies(rot), 1.0, layout)
        y, error = y.cpu().numpy(), (TURN * size).cpu().numpy()
        scale = np.maximum(np.abs(y).max(-1) / float(QMAX[cell]), 2.0 ** -100)
        assert np.all(np.abs(turned[0][1] - scale) <= 2.0 ** -16 * scale)
        r, off = np.abs(y) / scale[..., None], 2.0 ** -15 * np.abs(y) / scale[..., None] + 2 * error / scale[..., None]
        half = 0.5 if cell == INT8 else np.exp2(np.maximum(np.frexp(r + off)[1] - 1, -6) - 4.0)
        assert np.all(np.abs(turned[0][0] - y / scale[..., None]) <= half + off)


@pytest.mark.parametrize("cell", [E4M3, INT8])
def test_ties_one_by_one(cell):
    # all halves between neighbours of the format, both signs, under a maximum whose scale is 1
    if cell == INT8:
        halves = np.arange(-126.5, 127.0)
    else:
        grid = np.array(sorted({m * 2.0 ** e for e in range(-9, 6) for m in range(8 if e > -9 else 0, 16)} | {m * 2.0 ** -9 for m in range(8)}))
        grid = grid[grid <= 448]
        halves = (grid[1:] + grid[:-1]) / 2
        halves = np.concatenate([halves, -halves])
    assert nearest(halves.astype(np.float32), cell)[1].all()
    dim = 128
    rows = -(-len(halves) // (dim - 1))
    x = np.zeros((rows, dim), dtype=np.float32)
    x[:, 0] = QMAX[cell]
    x[:, 1:].reshape(-1)[:] = 0
    flat = np.zeros(rows * (dim - 1), dtype=np.float32)
    flat[:len(halves)] = halves
    x[:, 1:] = flat.reshape(rows, dim - 1)
    for kind in (F32, BF):
        v = torch.from_numpy(x).cuda().to(kind)[:, None]
        assert np.array_equal(v[:, 0].float().cpu().numpy(), x)
        cache, scale = torch.zeros(2, rows, 1, 1, dim, dtype=cell, device="cuda"), torch.zeros(2, rows, 1, 1, device="cuda")
        table, past = torch.arange(rows, dtype=torch.int32, device="cuda")[:, None], torch.zeros(rows, dtype=torch.int32, device="cuda")
        nf.kv_append(v, v, cache[0], cache[1], table, past, k_scale=scale[0], v_scale=scale[1])
        assert torch.all(scale == 1.0)
        for c in cache:
            assert np.array_equal(c[:, 0, 0].float().cpu().numpy(), nearest(x, cell)[0])
