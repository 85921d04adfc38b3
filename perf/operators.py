"""The library's token-side operators as a user calls them, with their plain forms.

Five operators: RMSNorm with an 8-bit output and its scales (with or without the residual's addition), the embedding
lookup with scaling, its gradient, the log probabilities of given tokens with entropy and top alternatives, and the
gradient of log probability and entropy.

A case is a dict of plain values.  ``prepare`` makes a case's inputs on the GPU from a seed, ``run`` makes one pass
over them -- through the library where ``own`` is true, in elementary torch operations where it is false -- and
``exact`` says in 64 bits what the pass returns.  ``work`` counts the bytes and operations a pass cannot do without.

Token ids are log-uniform over the vocabulary (density 1/id, as word frequencies fall off), a share of them padding
(id -1: a row of zeros, no gradient).  Logits are normal with a spread of 2.5, the given token raised in half of the
rows; masked entries are -inf, and where entries are masked the last row has nothing left.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
QMAX = {"e4m3": 448.0, "int8": 127.0}
SCALE_MIN = 2.0 ** -100  # smallest scale: that of a group of zeros can be divided by
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a decode step's rows, normalized for an 8-bit projection; one scale for each token
        {"name": "norm q8 decode 16x4096", "op": "norm_q8", "rows": 16, "hidden": 4096, "residual": True, "fmt": "e4m3", "group": 0},
        # a block's first norm in 8-bit integers, a medium batch
        {"name": "norm q8 int8 4096x5120", "op": "norm_q8", "rows": 4096, "hidden": 5120, "residual": False, "fmt": "int8", "group": 0},
        # a prefill batch, one scale for each 128 columns
        {"name": "norm q8 prefill 16384x8192", "op": "norm_q8", "rows": 16384, "hidden": 8192, "residual": True, "fmt": "e4m3", "group": 128},
        # the tokens of a decode step
        {"name": "embed decode 64x4096", "op": "embed", "tokens": 64, "hidden": 4096, "vocab": 131072, "scale": 1.0, "pad": 0.0},
        # a training batch, the rows scaled by sqrt(hidden), some padding
        {"name": "embed train 32768x8192", "op": "embed", "tokens": 32768, "hidden": 8192, "vocab": 131072, "scale": 90.5, "pad": 0.03},
        # short sequences added into the 16-bit gradient that the output layer has written
        {"name": "embed grad 2000x2048 add", "op": "embed_grad", "tokens": 2000, "hidden": 2048, "vocab": 32003, "scale": 45.25, "pad": 0.1, "grad": "bf16", "add": True},
        # a training batch, the whole table's gradient written
        {"name": "embed grad 16384x4096", "op": "embed_grad", "tokens": 16384, "hidden": 4096, "vocab": 131072, "scale": 1.0, "pad": 0.0, "grad": "f32", "add": False},
        # a decode step that answers with the alternatives
        {"name": "logprob decode 16x131072", "op": "logprob", "rows": 16, "vocab": 131072, "type": "bf16", "temperature": 1.0, "top": 5, "mask": 0.0},
        # scoring given answers with alternatives, an odd vocabulary in fp32
        {"name": "logprob 1000x100003 f32", "op": "logprob", "rows": 1000, "vocab": 100003, "type": "f32", "temperature": 0.8, "top": 20, "mask": 0.0},
        # scoring a batch of rollouts
        {"name": "logprob 8192x131072", "op": "logprob", "rows": 8192, "vocab": 131072, "type": "bf16", "temperature": 1.0, "top": 0, "mask": 0.0},
        # the policy gradient's step back to the logits, with an entropy term
        {"name": "logprob grad 4096x131072", "op": "logprob_grad", "rows": 4096, "vocab": 131072, "type": "bf16", "temperature": 1.0, "entropy": True, "mask": 0.0},
        # a small batch's step back in fp32, a restricted vocabulary
        {"name": "logprob grad 300x32003 f32", "op": "logprob_grad", "rows": 300, "vocab": 32003, "type": "f32", "temperature": 0.8, "entropy": False, "mask": 0.3},
    ]


def _log(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["norm_q8", "embed", "embed_grad", "logprob", "logprob_grad"])
    if op == "norm_q8":
        return {"op": op, "rows": _log(rng, 1, 16384), "hidden": 8 * _log(rng, 32, 1024), "residual": rng.random() < 0.6,
                "fmt": rng.choice(["e4m3", "e4m3", "int8"]), "group": rng.choice([0, 0, 128])}
    if op == "embed":
        return {"op": op, "tokens": _log(rng, 1, 32768), "hidden": 8 * _log(rng, 8, 1024), "vocab": _log(rng, 1000, 131072),
                "scale": round(rng.uniform(0.5, 90.0), 2), "pad": rng.choice([0.0, 0.1])}
    if op == "embed_grad":
        hidden = 8 * _log(rng, 8, 512)
        return {"op": op, "tokens": _log(rng, 1, 65536), "hidden": hidden, "vocab": _log(rng, 1000, 131072), "scale": round(rng.uniform(0.5, 64.0), 2),
                "pad": rng.choice([0.0, 0.1]), "grad": rng.choice(["f32", "bf16"]), "add": rng.random() < 0.5}
    rows, kind = _log(rng, 1, 4096), rng.choice(["bf16", "f32"])
    vocab = min(_log(rng, 1000, 160000), max(1000, 500_000_000 // rows))
    c = {"op": op, "rows": rows, "vocab": vocab, "type": kind, "temperature": round(rng.uniform(0.5, 1.5), 2), "mask": rng.choice([0.0, 0.0, 0.4])}
    c.update({"top": rng.choice([0, 1, 5, 20, 32])} if op == "logprob" else {"entropy": rng.random() < 0.5})
    return c


def _ids(g, n, vocab, pad):
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(vocab + 1.0)).long() - 1).clamp(0, vocab - 1)
    return torch.where(torch.rand(n, generator=g, device="cuda") < pad, -1, ids) if pad else ids


def _logits(g, case):
    rows, vocab = case["rows"], case["vocab"]
    targets = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    logits = torch.randn(rows, vocab, generator=g, device="cuda").mul_(2.5)
    up = torch.where(torch.rand(rows, 1, generator=g, device="cuda") < 0.5, 14.0, 0.0)
    logits.scatter_add_(1, targets[:, None], up)
    if case["mask"]:
        gone = torch.rand(rows, vocab, generator=g, device="cuda") < case["mask"]
        gone[-1] = True
        logits.masked_fill_(gone, -math.inf)
    return logits.to(TYPES[case["type"]]), targets


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], dict(case)
    if op == "norm_q8":
        shape = (case["rows"], case["hidden"])
        s["x"] = torch.randn(shape, generator=g, device="cuda").bfloat16()
        s["weight"] = (1 + 0.1 * torch.randn(case["hidden"], generator=g, device="cuda")).bfloat16()
        s["res"] = torch.randn(shape, generator=g, device="cuda").mul_(4).bfloat16() if case["residual"] else None
    elif op == "embed":
        s["ids"] = _ids(g, case["tokens"], case["vocab"], case["pad"])
        s["table"] = torch.randn(case["vocab"], case["hidden"], generator=g, device="cuda").mul_(0.02).bfloat16()
    elif op == "embed_grad":
        s["ids"] = _ids(g, case["tokens"], case["vocab"], case["pad"])
        s["dy"] = torch.randn(case["tokens"], case["hidden"], generator=g, device="cuda").mul_(0.01).bfloat16()
        s["grad_now"] = torch.randn(case["vocab"], case["hidden"], generator=g, device="cuda").mul_(0.01).to(TYPES[case["grad"]]) if case["add"] else None
    else:
        s["logits"], s["targets"] = _logits(g, case)
        if op == "logprob_grad":  # what the forward pass has saved, and the loss's gradients
            _, s["ent"], s["stats"] = _logprob(s["logits"], s["targets"], case["temperature"])
            s["d_logprob"] = torch.randn(case["rows"], generator=g, device="cuda")
            s["d_entropy"] = torch.randn(case["rows"], generator=g, device="cuda").mul_(0.01) if case["entropy"] else None
    return s


# ---- the plain forms

def _norm_q8(x, residual, weight, fmt, group):
    rows, hidden = x.shape
    v = x.float()
    if residual is not None:
        v = v + residual.float()
        residual.copy_(v)
    y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * weight.float()
    width = group or hidden
    groups = -(-hidden // width)
    y = torch.nn.functional.pad(y, (0, groups * width - hidden)).view(rows, groups, width)
    scale = (y.abs().amax(2) / QMAX[fmt]).clamp(min=SCALE_MIN)
    q = torch.where(scale.isfinite()[..., None], y / scale[..., None], 0.0).clamp(-QMAX[fmt], QMAX[fmt]).view(rows, -1)[:, :hidden]
    q = q.to(torch.float8_e4m3fn) if fmt == "e4m3" else q.round().to(torch.bfloat16)
    return q.contiguous(), scale if group else scale.view(rows)


def _embed(ids, table, scale):
    rows = table[ids.clamp(min=0)].float() * scale
    return torch.where((ids >= 0)[:, None], rows, 0.0).to(table.dtype)


def _embed_grad(dy, ids, vocab, scale, grad, kind):
    keep = ids >= 0
    sums = torch.zeros(vocab, dy.shape[1], device="cuda")
    sums.index_add_(0, ids.clamp(min=0), torch.where(keep[:, None], dy.float() * scale, 0.0))
    if grad is None:
        return sums.to(kind)
    grad.copy_(grad.float() + sums)
    return grad


def _logprob(logits, targets, temperature):
    l = logits.float()
    m = l.amax(1, keepdim=True)
    z = (l - torch.where(m > -math.inf, m, 0.0)) / temperature
    p = torch.exp(z)
    total = p.sum(1, keepdim=True)
    log_total = torch.log(total)
    logprob = (z.gather(1, targets[:, None]) - log_total).squeeze(1)
    logprob = torch.where(m[:, 0] > -math.inf, logprob, -math.inf)
    entropy = log_total - torch.where(p > 0, p * z, 0.0).sum(1, keepdim=True) / total
    entropy = torch.where(m > -math.inf, entropy, 0.0).squeeze(1)
    return logprob, entropy, torch.cat([m, log_total], 1)


def _top(logits, stats, temperature, top):
    l = logits.float()
    bits = l.view(torch.int32).long()
    order = torch.where(bits < 0, ~(bits & 0x7FFFFFFF), bits)  # grows with the value; a tie goes to the lower index
    key = (order << 32) | (0xFFFFFFFF - torch.arange(l.shape[1], device="cuda"))
    at = torch.topk(key, min(top, l.shape[1]), dim=1).indices
    best = l.gather(1, at)
    here = best > -math.inf
    return torch.where(here, (best - stats[:, :1]) / temperature - stats[:, 1:], -math.inf), torch.where(here, at, -1)


def _logprob_grad(logits, targets, stats, entropy, d_logprob, d_entropy, temperature):
    l, m = logits.float(), stats[:, :1]
    log_p = torch.where(l > -math.inf, (l - torch.where(m > -math.inf, m, 0.0)) / temperature - torch.where(m > -math.inf, stats[:, 1:], 0.0), -math.inf)
    p = torch.exp(log_p)
    g = -d_logprob[:, None] * p
    if d_entropy is not None:
        g -= d_entropy[:, None] * torch.where(p > 0, p * (log_p + entropy[:, None]), 0.0)
    g.scatter_add_(1, targets[:, None], torch.where(m > -math.inf, d_logprob[:, None], 0.0))
    return (g / temperature).to(logits.dtype)


def _plain(s):
    op = s["op"]
    if op == "norm_q8":
        q, scale = _norm_q8(s["x"], s["res"], s["weight"], s["fmt"], s["group"])
        return {"q": q, "scale": scale, "residual": s["res"]}
    if op == "embed":
        return {"y": _embed(s["ids"], s["table"], s["scale"])}
    if op == "embed_grad":
        return {"grad": _embed_grad(s["dy"], s["ids"], s["vocab"], s["scale"], s["grad_now"], TYPES[s["grad"]])}
    if op == "logprob":
        logprob, entropy, stats = _logprob(s["logits"], s["targets"], s["temperature"])
        top = _top(s["logits"], stats, s["temperature"], s["top"]) if s["top"] else (None, None)
        return {"logprob": logprob, "entropy": entropy, "stats": stats, "top": top[0], "top_ids": top[1]}
    return {"dlogits": _logprob_grad(s["logits"], s["targets"], s["stats"], s["ent"], s["d_logprob"], s["d_entropy"], s["temperature"])}


def _library(s):
    import row_normalization_inner_gb300 as nf
    op = s["op"]
    if op == "norm_q8":
        if s["res"] is None:
            q, scale = nf.rmsnorm_q8(s["x"], s["weight"], EPS, fmt=s["fmt"], group=s["group"])
        else:
            q, scale = nf.fused_add_rmsnorm_q8(s["x"], s["res"], s["weight"], EPS, fmt=s["fmt"], group=s["group"])
        # the 8-bit integers as the numbers they stand for (exact in bf16); e4m3 is a floating type already
        return {"q": q if s["fmt"] == "e4m3" else q.to(torch.bfloat16), "scale": scale, "residual": s["res"]}
    if op == "embed":
        return {"y": nf.embedding_fwd(s["ids"], s["table"], s["scale"])}
    if op == "embed_grad":
        return {"grad": nf.embedding_bwd(s["dy"], s["ids"], s["vocab"], s["scale"], dtype=TYPES[s["grad"]], accumulate=s["grad_now"])}
    if op == "logprob":
        logprob, entropy, stats, top, top_ids = nf.token_logprob_fwd(s["logits"], s["targets"], s["temperature"], top=s["top"])
        return {"logprob": logprob, "entropy": entropy, "stats": stats, "top": top, "top_ids": top_ids}
    return {"dlogits": nf.token_logprob_bwd(s["logits"], s["targets"], s["stats"], s["ent"], s["d_logprob"], s["d_entropy"], s["temperature"])}


def run(state):
    return _library(state) if own else _plain(state)


# ---- what a pass cannot do without

def _unique(n, vocab):
    """Expected number of distinct ids among n of _ids()."""
    k = np.arange(vocab, dtype=np.float64)
    share = np.log((k + 2) / (k + 1)) / math.log(vocab + 1.0)
    return float(np.sum(-np.expm1(n * np.log1p(-share))))


def work(case):
    op = case["op"]
    if op == "norm_q8":
        n, h = case["rows"], case["hidden"]
        groups = -(-h // case["group"]) if case["group"] else 1
        return {"bytes": n * h * (7 if case["residual"] else 3) + 4 * n * groups + 2 * h, "flops": 7 * n * h}
    if op in ("embed", "embed_grad"):
        n, h, v = case["tokens"], case["hidden"], case["vocab"]
        kept = n * (1 - case["pad"])
        rows = _unique(kept, v)
        if op == "embed":
            return {"bytes": 8 * n + 2 * h * (rows + n), "flops": kept * h}
        size = 4 if case["grad"] == "f32" else 2
        return {"bytes": 8 * n + 2 * h * kept + size * h * (2 * rows if case["add"] else v), "flops": 2 * kept * h}
    n, v, size = case["rows"], case["vocab"], 2 if case["type"] == "bf16" else 4
    if op == "logprob":
        return {"bytes": n * v * size + n * (24 + 12 * case["top"]), "flops": 6 * n * v}
    return {"bytes": 2 * n * v * size + 28 * n, "flops": 6 * n * v}


# ---- in 64 bits, from the definitions

def _e4m3(v):
    """The nearest value of a format with 3 mantissa bits, smallest normal exponent -6 and largest value 448, ties to even."""
    a = v.abs().clamp(min=2.0 ** -40)
    step = torch.exp2(torch.floor(torch.log2(a)).clamp(min=-6.0) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_norm(s):
    x = s["x"].double()
    v = x if s["res"] is None else x + s["res"].double()
    rows, hidden = v.shape
    rms = torch.linalg.vector_norm(v, dim=1, keepdim=True).square().div(hidden).add(EPS).sqrt()
    y = v / rms * s["weight"].double()
    q, scales = torch.empty_like(y), []
    for at in range(0, hidden, s["group"] or hidden):
        part = slice(at, min(hidden, at + (s["group"] or hidden)))
        scale = torch.maximum(y[:, part].max(1).values, -y[:, part].min(1).values).div(QMAX[s["fmt"]]).clamp(min=SCALE_MIN)
        q[:, part] = _e4m3(y[:, part] / scale[:, None]) if s["fmt"] == "e4m3" else torch.round(y[:, part] / scale[:, None])
        scales.append(scale)
    return {"q": q, "scale": torch.stack(scales, 1) if s["group"] else scales[0], "residual": None if s["res"] is None else v}


def _exact_embed_grad(s):
    """Sums of equal ids as differences of running sums over the sorted tokens."""
    kept = torch.nonzero(s["ids"] >= 0)[:, 0]
    ids, order = torch.sort(s["ids"][kept])
    out = torch.zeros(s["vocab"], s["hidden"], device="cuda", dtype=torch.float64) if s["grad_now"] is None else s["grad_now"].double()
    if len(ids):
        last = torch.nonzero(torch.cat([ids[1:] != ids[:-1], ids.new_ones(1, dtype=torch.bool)]))[:, 0]
        for at in range(0, s["hidden"], 1024):
            run_sums = torch.cumsum(s["dy"][kept[order], at:at + 1024].double(), 0)[last]
            out[ids[last], at:at + 1024] += s["scale"] * torch.diff(run_sums, dim=0, prepend=run_sums.new_zeros(1, run_sums.shape[1]))
    return {"grad": out}


def _exact_rows(s):
    """Log probabilities, entropy and alternatives, or their gradient, some rows at a time."""
    parts, block = [], max(1, 50_000_000 // s["vocab"])
    for at in range(0, s["rows"], block):
        rows = slice(at, at + block)
        l, t = s["logits"][rows].double(), s["targets"][rows]
        z = l / s["temperature"]
        lse = torch.logsumexp(z, 1, keepdim=True)
        some = lse > -math.inf
        log_p = torch.where(some, z - lse, -math.inf)
        p = log_p.exp()
        h = -torch.xlogy(p, p).sum(1, keepdim=True)
        if s["op"] == "logprob":
            m = l.max(1, keepdim=True).values
            o = {"logprob": log_p.gather(1, t[:, None])[:, 0], "entropy": h[:, 0], "stats": torch.cat([m, torch.where(some, lse - m / s["temperature"], -math.inf)], 1)}
            if s["top"]:
                best, ids = torch.sort(log_p, dim=1, descending=True, stable=True)
                o["top"] = best[:, :s["top"]].clone()
                o["top_ids"] = torch.where(o["top"] > -math.inf, ids[:, :s["top"]], -1)
        else:
            g = -p * s["d_logprob"][rows].double()[:, None]
            g[torch.arange(len(t), device="cuda"), t] += s["d_logprob"][rows].double() * some[:, 0]
            if s["d_entropy"] is not None:
                g -= s["d_entropy"][rows].double()[:, None] * (torch.xlogy(p, p) + p * h)
            o = {"dlogits": g / s["temperature"]}
        parts.append(o)
    return {k: torch.cat([o[k] for o in parts]) for k in parts[0]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_q8":
        return _exact_norm(s)
    if case["op"] == "embed":
        out = s["table"].double().index_select(0, s["ids"].clamp(min=0)) * s["scale"]
        return {"y": out * (s["ids"] >= 0).double()[:, None]}
    if case["op"] == "embed_grad":
        return _exact_embed_grad(s)
    return _exact_rows(s)
