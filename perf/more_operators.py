"""The library's operators on attention heads as a user calls them, with their plain forms.

Five operators between a block's norm and its attention: the rotation of queries and keys by their positions and its
gradient, the RMSNorm of each query and key head with the rotation in the same pass and its gradient, and the step that
appends keys and values to a paged cache (rotating, and where wanted normalizing and quantizing, on the way).

A case is a dict of plain values.  ``prepare`` makes a case's inputs on the GPU from a seed, ``run`` makes one pass
over them -- through the library where ``own`` is true, in elementary torch operations where it is false -- and
``exact`` says in 64 bits what the pass returns.  ``work`` counts the bytes and operations a pass cannot do without.

Heads are normal; where ``fused`` is true they are views of one projection's output, [tokens, queries | keys | values],
as a user's program has them.  Positions count up from a start drawn below ``far``.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
BASE = 10000.0
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100  # smallest scale: that of a row of zeros can be divided by
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token for each of 16 sequences, 32 query and 8 key heads
        {"name": "rope decode 16x40x128", "op": "rope", "batch": 16, "tokens": 1, "q_heads": 32, "k_heads": 8, "dim": 128, "rot": 128, "layout": "half", "type": "bf16", "far": 4000, "scaling": "none", "fused": True},
        # far positions of a long document, half of the head rotated, frequencies scaled by parts, fp32
        {"name": "rope 1003x24x96 f32", "op": "rope", "batch": 1, "tokens": 1003, "q_heads": 20, "k_heads": 4, "dim": 96, "rot": 48, "layout": "interleaved", "type": "f32", "far": 1000000, "scaling": "parts", "fused": False},
        # a training batch, straight from the projection
        {"name": "rope train 4x4096x72x128", "op": "rope", "batch": 4, "tokens": 4096, "q_heads": 64, "k_heads": 8, "dim": 128, "rot": 128, "layout": "half", "type": "bf16", "far": 1, "scaling": "none", "fused": True},
        # a small batch's step back, as many key as query heads
        {"name": "rope grad 2x1023x32x64", "op": "rope_grad", "batch": 2, "tokens": 1023, "q_heads": 16, "k_heads": 16, "dim": 64, "rot": 64, "layout": "interleaved", "type": "bf16", "far": 1, "scaling": "none", "fused": False},
        # a training batch's step back
        {"name": "rope grad 2x8192x40x128", "op": "rope_grad", "batch": 2, "tokens": 8192, "q_heads": 32, "k_heads": 8, "dim": 128, "rot": 128, "layout": "half", "type": "bf16", "far": 1, "scaling": "linear", "fused": False},
        # a decode step with normalized heads
        {"name": "norm rope decode 64x48x128", "op": "norm_rope", "batch": 64, "tokens": 1, "q_heads": 40, "k_heads": 8, "dim": 128, "rot": 128, "layout": "half", "type": "bf16", "far": 30000, "scaling": "none", "fused": True},
        # a prefill batch, normalized and rotated
        {"name": "norm rope 16384x72x128", "op": "norm_rope", "batch": 1, "tokens": 16384, "q_heads": 64, "k_heads": 8, "dim": 128, "rot": 128, "layout": "half", "type": "bf16", "far": 1, "scaling": "ntk", "fused": True},
        # a small fp32 model's step back, heads of 80
        {"name": "norm rope grad 777x24x80 f32", "op": "norm_rope_grad", "batch": 1, "tokens": 777, "q_heads": 12, "k_heads": 12, "dim": 80, "rot": 80, "layout": "half", "type": "f32", "far": 1, "scaling": "none", "fused": False},
        # a training batch's step back with both weights' gradients
        {"name": "norm rope grad 4x4096x72x128", "op": "norm_rope_grad", "batch": 4, "tokens": 4096, "q_heads": 64, "k_heads": 8, "dim": 128, "rot": 128, "layout": "half", "type": "bf16", "far": 1, "scaling": "none", "fused": True},
        # one sequence's next token far into its context, an 8-bit cache
        {"name": "append 1x40x128 e4m3", "op": "append", "seqs": 1, "tokens": 1, "q_heads": 32, "k_heads": 8, "dim": 128, "rot": 128, "layout": "half", "type": "bf16", "far": 100000, "scaling": "parts", "norm": False, "cache": "e4m3", "page": 64},
        # a decode step of 128 sequences, normalized heads, pages of 16
        {"name": "append 128x40x128", "op": "append", "seqs": 128, "tokens": 128, "q_heads": 32, "k_heads": 8, "dim": 128, "rot": 128, "layout": "half", "type": "bf16", "far": 2000, "scaling": "none", "norm": True, "cache": "same", "page": 16},
        # chunks of 13 prompts of all lengths, an 8-bit cache
        {"name": "append chunks 8192x72x128 e4m3", "op": "append", "seqs": 13, "tokens": 8192, "q_heads": 64, "k_heads": 8, "dim": 128, "rot": 128, "layout": "half", "type": "bf16", "far": 3000, "scaling": "none", "norm": True, "cache": "e4m3", "page": 64},
    ]


def _log(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["rope", "rope_grad", "norm_rope", "norm_rope_grad", "append"])
    dim = rng.choice([64, 64, 80, 96, 112, 128, 128, 128, 192, 256])
    k_heads = _log(rng, 1, 16)
    c = {"op": op, "q_heads": k_heads * rng.choice([1, 1, 2, 4, 5, 8]), "k_heads": k_heads, "dim": dim,
         "rot": rng.choice([dim, dim, dim // 2]), "layout": rng.choice(["half", "half", "interleaved"]),
         "type": rng.choice(["bf16", "bf16", "bf16", "f32"]), "far": _log(rng, 1, 200000), "scaling": rng.choice(["none", "none", "linear", "ntk", "parts"])}
    size = 2 if c["type"] == "bf16" else 4
    most = 300_000_000 // ((c["q_heads"] + 2 * k_heads) * dim * size)  # a pass's heads in bytes: fewer than the largest listed case has
    if op == "append":
        tokens = _log(rng, 1, min(16384, most))
        seqs = tokens if rng.random() < 0.4 else _log(rng, 1, min(64, tokens))  # a decode step, or chunks
        # both caches hold 2^27 elements each at most
        far = max(1, min(c["far"], (1 << 27) // (seqs * k_heads * dim) - 256))
        return {**c, "far": far, "tokens": tokens, "seqs": seqs, "norm": rng.random() < 0.5, "cache": rng.choice(["same", "e4m3"]), "page": rng.choice([16, 16, 32, 64, 128, 100])}
    batch = _log(rng, 1, 64)
    return {**c, "batch": batch, "tokens": _log(rng, 1, max(1, min(16384, most) // batch)), "fused": rng.random() < 0.5}


def _frequencies(case):
    """Radians per position of each pair, with the scalings for contexts eight times as long as those of training."""
    rot, base, factor, length = case["rot"], BASE, 8.0, 8192.0
    if case["scaling"] == "ntk":
        base *= factor ** (rot / (rot - 2))
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "parts":
        keep = np.clip((length * f / (2 * math.pi) - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    return f


def _magnitude(case):
    return 0.1 * math.log(8.0) + 1.0 if case["scaling"] == "parts" else 1.0


def _heads(g, batch, tokens, counts, dim, kind, fused):
    if fused:
        all_heads = torch.randn(batch, tokens, sum(counts), dim, generator=g, device="cuda").to(kind)
        return list(torch.split(all_heads, counts, dim=2))
    return [torch.randn(batch, tokens, n, dim, generator=g, device="cuda").to(kind) for n in counts]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    f = _frequencies(case)
    s["frequencies"] = torch.from_numpy(f).cuda()
    # what the library rotates by: the share of a turn per position in units of 2^-64
    turns = [int(v / (2 * math.pi) * 2.0 ** 64) & (2 ** 64 - 1) for v in f.tolist()]
    s["rates"] = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device="cuda")
    kind, dim, hq, hk = TYPES[case["type"]], case["dim"], case["q_heads"], case["k_heads"]
    for name in ("q_weight", "k_weight"):
        s[name] = (1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).to(kind)
    if case["op"] == "append":
        return _prepare_append(s, case, g, kind)
    batch, tokens = case["batch"], case["tokens"]
    start = torch.randint(0, case["far"], (batch, 1), generator=g, device="cuda")
    s["positions"] = start + torch.arange(tokens, device="cuda")
    s["q"], s["k"] = _heads(g, batch, tokens, [hq, hk, hk], dim, kind, True)[:2] if case["fused"] else _heads(g, batch, tokens, [hq, hk], dim, kind, False)
    if case["op"].endswith("grad"):  # of the rotated heads, as attention's backward pass leaves them
        s["dq"], s["dk"] = [t.mul_(0.01) for t in _heads(g, batch, tokens, [hq, hk], dim, kind, False)]
    return s


def _prepare_append(s, case, g, kind):
    seqs, tokens, page, dim, hk = case["seqs"], case["tokens"], case["page"], case["dim"], case["k_heads"]
    s["q"], s["k"], s["v"] = [t[0] for t in _heads(g, 1, tokens, [case["q_heads"], hk, hk], dim, kind, True)]
    # lengths before the step, and where each sequence's new tokens begin
    s["past"] = torch.randint(case["far"] // 2, case["far"], (seqs,), generator=g, device="cuda", dtype=torch.int32)
    new = torch.ones(seqs, dtype=torch.int64, device="cuda")
    s["starts"] = None
    if tokens > seqs:
        cuts = torch.sort(torch.randperm(tokens - 1, generator=g, device="cuda")[:seqs - 1] + 1).values
        starts = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), tokens)])
        new = torch.diff(starts)
        s["starts"] = starts.int()
    # pages in any order, those of a sequence up to its last token; some of the cache's are free
    most = -(-(case["far"] + (tokens - seqs + 1)) // page)
    pages = (seqs * (case["far"] - 1) + tokens) // page + seqs
    held = -(-(s["past"] + new) // page)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    at = torch.cumsum(held, 0) - held
    column = torch.arange(most, device="cuda")
    s["table"] = torch.where(column < held[:, None], order[(at[:, None] + column).clamp(max=pages - 1)], -1).int()
    shape = (pages, page, hk, dim)
    s["k_scale"] = s["v_scale"] = None
    for name in ("k", "v"):
        cache = torch.randn(shape, generator=g, device="cuda").mul_(16.0 if case["cache"] == "e4m3" else 1.0)
        s[name + "_cache"] = cache.to(torch.float8_e4m3fn if case["cache"] == "e4m3" else kind)
        if case["cache"] == "e4m3":
            s[name + "_scale"] = torch.rand(shape[:3], generator=g, device="cuda") * 0.02
    return s


# ---- the plain forms

def _rotate(x, positions, frequencies, magnitude, layout, back=False):
    """Heads [..., heads, dim] in fp32, their first 2 * len(frequencies) elements rotated by each token's angles."""
    angle = positions.double()[..., None, None] * frequencies
    cos, sin = (torch.cos(angle) * magnitude).float(), (torch.sin(angle) * (-magnitude if back else magnitude)).float()
    n = len(frequencies)
    if layout == "half":
        a, b = x[..., :n], x[..., n:2 * n]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * n:]], -1)


def _norm(x, weight):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()


def _norm_grad(dy, x, weight):
    x = x.float()
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * rstd
    g = dy * weight.float()
    dx = rstd * (g - n * (g * n).mean(-1, keepdim=True))
    return dx, (dy * n).flatten(0, -2).sum(0)


def _quantize(y):
    top = y.abs().amax(-1)
    scale = torch.where(top.isfinite(), (top / E4M3_MAX).clamp(min=SCALE_MIN), math.nan)
    q = torch.where(scale.isfinite()[..., None], y / scale[..., None], 0.0).clamp(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn), scale


def _append(s):
    tokens, kind = s["tokens"], s["k"].dtype
    i = torch.arange(tokens, device="cuda")
    seq, begin = i, i
    if s["starts"] is not None:
        seq = torch.searchsorted(s["starts"].long(), i, right=True) - 1
        begin = s["starts"].long()[seq]
    positions = s["past"].long()[seq] + i - begin
    page, slot = s["table"].long()[seq, positions // s["page"]], positions % s["page"]
    q, k = s["q"].float(), s["k"].float()
    if s["norm"]:
        q, k = _norm(q, s["q_weight"]), _norm(k, s["k_weight"])
    q, k = (_rotate(t, positions, s["frequencies"], _magnitude(s), s["layout"]) for t in (q, k))
    if s["cache"] == "same":
        s["k_cache"][page, slot] = k.to(kind)
        s["v_cache"][page, slot] = s["v"]
    else:
        for name, rows in (("k", k), ("v", s["v"].float())):
            values, scale = _quantize(rows)
            s[name + "_cache"].view(torch.uint8)[page, slot] = values.view(torch.uint8)
            s[name + "_scale"][page, slot] = scale
    return {"q": q.to(kind), **_cache(s)}


def _cache(s):
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _plain(s):
    op = s["op"]
    if op == "append":
        return _append(s)
    rotate = lambda t, back=False: _rotate(t.float(), s["positions"], s["frequencies"], _magnitude(s), s["layout"], back)  # noqa: E731
    if op == "rope":
        return {n: rotate(s[n]).to(s[n].dtype) for n in ("q", "k")}
    if op == "rope_grad":
        return {n: rotate(s["d" + n], True).to(s[n].dtype) for n in ("q", "k")}
    if op == "norm_rope":
        return {n: rotate(_norm(s[n].float(), s[n + "_weight"])).to(s[n].dtype) for n in ("q", "k")}
    dq, dq_weight = _norm_grad(rotate(s["dq"], True), s["q"], s["q_weight"])
    dk, dk_weight = _norm_grad(rotate(s["dk"], True), s["k"], s["k_weight"])
    return {"q": dq.to(s["q"].dtype), "k": dk.to(s["k"].dtype), "q_weight": dq_weight, "k_weight": dk_weight}


def _library(s):
    import row_normalization_inner_gb300 as nf
    op, how = s["op"], {"layout": s["layout"], "magnitude": _magnitude(s)}
    if op == "append":
        weights = {"q_weight": s["q_weight"], "k_weight": s["k_weight"], "eps": EPS} if s["norm"] else {}
        q = nf.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["past"], starts=s["starts"], rates=s["rates"],
                         q=s["q"], k_scale=s["k_scale"], v_scale=s["v_scale"], **weights, **how)
        return {"q": q, **_cache(s)}
    if op == "rope":
        q, k = nf.rope_fwd(s["q"], s["k"], s["positions"], s["rates"], **how)
    elif op == "rope_grad":
        q, k = nf.rope_bwd(s["dq"], s["dk"], s["positions"], s["rates"], **how)
    elif op == "norm_rope":
        q, k = nf.qk_rmsnorm_rope_fwd(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["rates"], eps=EPS, **how)
    else:
        q, k, q_weight, k_weight = nf.qk_rmsnorm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"],
                                                          s["rates"], eps=EPS, **how)
        return {"q": q, "k": k, "q_weight": q_weight, "k_weight": k_weight}
    return {"q": q, "k": k}


def run(state):
    return _library(state) if own else _plain(state)


# ---- what a pass cannot do without

def work(case):
    op, dim, size = case["op"], case["dim"], 2 if case["type"] == "bf16" else 4
    hq, hk = case["q_heads"], case["k_heads"]
    turn, norm = 3 * case["rot"], 4 * dim
    if op == "append":
        n, cell = case["tokens"], 1 if case["cache"] == "e4m3" else size
        stored = 2 * hk * (dim * cell + (4 if case["cache"] == "e4m3" else 0))
        pages = case["seqs"] + n // case["page"]
        flops = (hq + hk) * (turn + (norm if case["norm"] else 0)) + (2 * hk * 2 * dim if case["cache"] == "e4m3" else 0)
        return {"bytes": n * ((2 * hq + 2 * hk) * dim * size + stored) + 4 * pages + 8 * case["seqs"] + 4 * case["rot"], "flops": n * flops}
    n, rows = case["batch"] * case["tokens"], case["batch"] * case["tokens"] * (hq + hk)
    if op in ("rope", "rope_grad"):
        return {"bytes": 2 * rows * dim * size + 8 * n + 4 * case["rot"], "flops": rows * turn}
    if op == "norm_rope":
        return {"bytes": 2 * rows * dim * size + 8 * n + 4 * case["rot"] + 2 * dim * size, "flops": rows * (turn + norm)}
    return {"bytes": 3 * rows * dim * size + 8 * n + 4 * case["rot"] + 2 * dim * (size + 4), "flops": rows * (turn + 3 * norm)}


# ---- in 64 bits, from the definitions

def _turn(case, positions):
    """The rotation of each token as complex numbers of length `magnitude`, [..., 1, pairs]."""
    angle = torch.remainder(positions.double()[..., None, None] * torch.from_numpy(_frequencies(case)).cuda(), 2 * math.pi)
    return torch.polar(torch.full_like(angle, _magnitude(case)), angle)


def _turned(case, x, z):
    n = z.shape[-1]
    y = x.double().clone()
    if case["layout"] == "half":
        w = torch.complex(y[..., :n].contiguous(), y[..., n:2 * n].contiguous()) * z
        y[..., :n], y[..., n:2 * n] = w.real, w.imag
    else:
        w = torch.view_as_complex(y[..., :2 * n].reshape(*y.shape[:-1], n, 2)) * z
        y[..., :2 * n] = torch.view_as_real(w).flatten(-2)
    return y


def _unit(x):
    """Heads over their root mean square, and that root."""
    rms = (torch.linalg.vector_norm(x.double(), dim=-1, keepdim=True).square() / x.shape[-1] + EPS).sqrt()
    return x.double() / rms, rms


def _e4m3(v):
    """The nearest value of a format with 3 mantissa bits, smallest normal exponent -6 and largest value 448, ties to even."""
    a = v.abs().clamp(min=2.0 ** -40)
    step = torch.exp2(torch.floor(torch.log2(a)).clamp(min=-6.0) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_append(case, s):
    starts = s["starts"].tolist() if s["starts"] is not None else list(range(case["seqs"] + 1))
    past = s["past"].tolist()
    positions = torch.cat([torch.arange(past[n], past[n] + starts[n + 1] - starts[n]) for n in range(case["seqs"])]).cuda()
    seq = torch.repeat_interleave(torch.arange(case["seqs"]), torch.diff(torch.tensor(starts))).cuda()
    # the flat slot of each token
    slots = s["table"].long().flatten()[seq * s["table"].shape[1] + torch.div(positions, case["page"], rounding_mode="floor")] * case["page"] + positions % case["page"]
    z = _turn(case, positions)
    q, k = s["q"], s["k"]
    if case["norm"]:
        q, k = _unit(q)[0] * s["q_weight"].double(), _unit(k)[0] * s["k_weight"].double()
    out = {"q": _turned(case, q, z)}
    for name, rows in (("k", _turned(case, k, z)), ("v", s["v"].double())):
        cache = s[name + "_cache"].to(torch.float64).flatten(0, 1)
        out[name + "_scale"] = None
        if case["cache"] == "e4m3":
            scale = torch.maximum(rows.max(-1).values, -rows.min(-1).values).div(E4M3_MAX).clamp(min=SCALE_MIN)
            rows = _e4m3(rows / scale[..., None])
            out[name + "_scale"] = s[name + "_scale"].double().flatten(0, 1).index_copy(0, slots, scale).view(s[name + "_scale"].shape)
        out[name + "_cache"] = cache.index_copy(0, slots, rows).view(s[name + "_cache"].shape)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return _exact_append(case, s)
    z = _turn(case, s["positions"])
    if op == "rope":
        return {n: _turned(case, s[n], z) for n in ("q", "k")}
    if op == "rope_grad":  # the transpose of a rotation turns back
        return {n: _turned(case, s["d" + n], z.conj()) for n in ("q", "k")}
    if op == "norm_rope":
        return {n: _turned(case, _unit(s[n])[0] * s[n + "_weight"].double(), z) for n in ("q", "k")}
    out = {}
    for n in ("q", "k"):  # the norm's gradient removes the part along the head
        dy, (unit, rms) = _turned(case, s["d" + n], z.conj()), _unit(s[n])
        out[n + "_weight"] = torch.einsum("...d,...d->d", dy, unit)
        g = dy * s[n + "_weight"].double()
        out[n] = (g - unit * torch.einsum("...d,...d->...", g, unit)[..., None] / case["dim"]) / rms
    return out
