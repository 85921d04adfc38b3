"""The operators on attention heads in 64 bits, with bounds on what fp32 kernels may be off.

Bounds.  u = 2^-24 is half a step of fp32.  An angle is a 64-bit integer
rounded to fp32 (u relative, at most pi u in radians), its sine and cosine are
within 2 u each and take the magnitude with one more rounding; a turned element
m (x c - y s) therefore is within 8 u m (|x| + |y|), products and their sum
included: TURN = 2^-21 of m (|x| + |y|).  A normalized element carries the sum
of squares (nonnegative terms, at most 64 additions in a chain: 64 u, halved by
the root), an rsqrt within 4 u and four products: 2^-18 relative, NORM, covers
it.  Both together stay below 2^-17 m (|x| + |y|).
"""
import math

import torch

TURN = 2.0 ** -21
NORM = 2.0 ** -18
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def frequencies(dim, base=10000.0):
    return torch.tensor([base ** (-2 * i / dim) for i in range(dim // 2)], dtype=torch.float64)


def pairs_of(dim, rot, layout):
    """Indices of the pairs' first and second elements, and of the rest."""
    i = torch.arange(rot // 2)
    a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    return a, b, torch.arange(rot, dim)


def turn(x, positions, freq, magnitude=1.0, layout="half", back=False):
    """(turned heads, the sums m (|x| + |y|) of each element's pair; |x| where it is not turned)."""
    x = x.double()
    a, b, _ = pairs_of(x.shape[-1], 2 * len(freq), layout)
    a, b = a.to(x.device), b.to(x.device)
    angle = positions.double()[..., None, None] * freq.to(x.device)
    c, s = torch.cos(angle) * magnitude, torch.sin(angle) * magnitude * (-1 if back else 1)
    y, size = x.clone(), x.abs()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    both = magnitude * (x[..., a].abs() + x[..., b].abs())
    size[..., a], size[..., b] = both, both
    return y, size


def normed(x, w, eps):
    x = x.double()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()


def close(got, ref, error, kind=None):
    """got within `error` of ref before its one rounding."""
    h = HALF_STEP[kind or got.dtype]
    off = (got.double() - ref).abs()
    tol = h * ref.abs() + (1 + h) * error + 2.0 ** -133
    bad = ~(off <= tol)
    assert not bad.any(), (int(bad.sum()), bad.numel(), off[bad][:4], ref[bad][:4], tol[bad][:4])


def norm_turn_grad(dy, x, w, eps, positions, freq, magnitude=1.0, layout="half"):
    """(dx, dw, bound of dx, bound of dw) in 64 bits.

    g is within TURN of its pair's size G >= |g|; every product, the mean and
    rstd add less than 2^-18 relative to sums of absolute values, so dx is
    within 2^-17 rstd (G |w| + |n| mean(G |w n|)).  A row's term of dw is within
    2^-17 G |n|; their sum adds at most (48 + rows / 2000) u of the sum of
    |g n| (a warp's rows in a chain, 2432 warps at most; the warp, the CTA, 608
    CTAs in 32 chains and these)."""
    g, size = turn(dy, positions, freq, magnitude, layout, back=True) if freq is not None else (dy.double(), dy.double().abs())
    x, w = x.double(), w.double()
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * rstd
    dx = rstd * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    dx_off = 2.0 ** -17 * rstd * (size * w.abs() + n.abs() * (size * (w * n).abs()).mean(-1, keepdim=True))
    rows = x.numel() // max(1, x.shape[-1])
    terms = (size * n.abs()).flatten(0, -2).sum(0)
    return dx, (g * n).flatten(0, -2).sum(0), dx_off, terms * (2.0 ** -17 + (48 + rows / 2000) * 2.0 ** -24)


def check_quantized(q, scale, y, error):
    """8-bit rows and their scales: a row's largest |y| is at least half of any pair's size, so the scale is within
    2^-16; q is the nearest value of y / scale."""
    top = QMAX[q.dtype]
    ref = (y.abs().amax(-1) / top).clamp(min=2.0 ** -100)
    assert torch.all((scale.double() - ref).abs() <= 2.0 ** -16 * ref)
    v = y / ref[..., None]
    half = torch.full_like(v, 0.5) if q.dtype == torch.int8 else torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10)
    off = (q.to(torch.float32).double() - v).abs()
    bad = ~(off <= half + 2.0 ** -15 * v.abs() + 2 * error / ref[..., None])
    assert not bad.any(), (int(bad.sum()), off[bad][:4], v[bad][:4])
    assert torch.all(q.to(torch.float32).abs() <= top)


def heads(generator, *shape, kind=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=generator, device="cuda") * scale).to(kind)


def fused_views(generator, batch, tokens, counts, dim, kind):
    """Queries, keys and values as views of one projection's output."""
    whole = heads(generator, batch, tokens, sum(counts), dim, kind=kind)
    return whole, list(torch.split(whole, counts, 2))


def rates_of(rot, **kw):
    import row_normalization_inner_gb300 as nf
    return nf.rope_rates(rot, **kw) if rot else None


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


assert math.isclose(TURN, 8 * 2.0 ** -24)
