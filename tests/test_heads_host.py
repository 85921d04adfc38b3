"""Host-side tests of the operators on attention heads (no GPU needed): rates,
and arguments that are refused before anything is launched."""
import ctypes
import math

import numpy as np
import pytest
import torch

import row_normalization_inner_gb300 as nf

# Fake, never dereferenced addresses, far enough apart for the sizes below.
A, B, C, D, E, F, G, H, I, J, K, L = (k << 36 for k in range(1, 13))
BIG = 1 << 41


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    yield


# ---------------------------------------------------------------- rates

def turns(rates):
    return np.array([int(r) & (2 ** 64 - 1) for r in rates.tolist()], dtype=object) / 2 ** 64


def test_rates_are_shares_of_a_turn():
    for dim in (2, 64, 128, 20, 512):
        f = np.array([10000.0 ** (-2 * i / dim) for i in range(dim // 2)])
        got = turns(nf.rope_rates(dim, device="cpu")).astype(float)
        # three roundings of 2^-53 in the frequency, one in 2 pi, one in the quotient; half a step of the rate
        assert np.all(np.abs(got - f / (2 * math.pi)) <= 8 * 2.0 ** -53 * f + 2.0 ** -65)


def test_scalings():
    dim, s, length = 64, 8.0, 4096.0
    f = np.array([500000.0 ** (-2 * i / dim) for i in range(dim // 2)])
    make = lambda **kw: turns(nf.rope_rates(dim, 500000.0, device="cpu", **kw)).astype(float) * 2 * math.pi  # noqa: E731
    # roundings of the powers, and half a step of the rates themselves: 2^-65 turns
    tol = 2.0 ** -48 * f + 2.0 ** -65 * 2 * math.pi
    assert np.all(np.abs(make(scaling="linear", factor=s) - f / s) <= tol)
    ntk = np.array([(500000.0 * s ** (dim / (dim - 2))) ** (-2 * i / dim) for i in range(dim // 2)])
    assert np.all(np.abs(make(scaling="ntk", factor=s) - ntk) <= tol)
    assert abs(ntk[-1] / (f[-1] / s) - 1) < 1e-12  # the slowest pair is slowed by the factor
    got = make(scaling="parts", factor=s, length=length, low=1.0, high=4.0)
    per_context = length * f / (2 * math.pi)
    fast, slow = per_context >= 4.0, per_context <= 1.0
    assert fast.any() and slow.any() and (~fast & ~slow).any()
    assert np.all(np.abs(got[fast] - f[fast]) <= tol[fast]) and np.all(np.abs(got[slow] - f[slow] / s) <= tol[slow])
    keep = (per_context - 1.0) / 3.0
    mixed = ~fast & ~slow
    assert np.all(np.abs(got - f * (keep + (1 - keep) / s))[mixed] <= 16 * tol[mixed])
    assert np.array_equal(nf.rope_rates(dim, 500000.0, device="cpu", scaling="parts", factor=1.0, length=length).numpy(),
                          nf.rope_rates(dim, 500000.0, device="cpu").numpy())


def test_given_frequencies():
    f = [1.0, -1.0, 2 * math.pi, 0.0, 1e-9, 1000.0, -1e-300, 1e-4]
    got = nf.rope_rates(16, frequencies=f, device="cpu")
    t = turns(got).astype(float)
    off = np.abs(t - np.array([x / (2 * math.pi) % 1.0 for x in f]))
    assert np.all(np.minimum(off, 1 - off) <= 1e-13)  # modulo a turn
    assert int(got[3]) == 0 and int(got[6]) == 0
    # the other way round is the same rate, to the last bit
    assert torch.equal(nf.rope_rates(16, frequencies=[-x for x in f], device="cpu"), -got)
    # small rates keep their digits: a share of a turn has 64 bits behind the point
    assert abs(t[4] / (1e-9 / (2 * math.pi)) - 1) < 2.0 ** -32


def test_rates_refusals():
    r = (ctypes.c_uint64 * 256)()
    ok = dict(rates=r, dim=64, base=1e4, scaling=0, factor=1.0, length=1.0, low=1.0, high=2.0)
    assert nf.nf_rope_rates(*ok.values()) == nf.NF_OK
    inf, nan = math.inf, math.nan
    for bad in ({"rates": None}, {"dim": 0}, {"dim": 63}, {"dim": 514}, {"dim": -2}, {"base": 1.0}, {"base": nan}, {"base": inf}, {"scaling": 4},
                {"scaling": -1}, {"scaling": 1, "factor": 0.5}, {"scaling": 1, "factor": nan}, {"scaling": 2, "dim": 2},
                {"scaling": 2, "factor": 1e300}, {"scaling": 3, "length": 0.0}, {"scaling": 3, "length": inf}, {"scaling": 3, "low": -1.0},
                {"scaling": 3, "low": 2.0}, {"scaling": 3, "high": nan}):
        assert nf.nf_rope_rates(*(ok | bad).values()) == nf.NF_ERR_INVALID_ARG, bad
    f = (ctypes.c_double * 4)(1.0, 2.0, nan, 0.0)
    assert nf.nf_rope_rates_of(r, f, 2) == nf.NF_OK
    assert nf.nf_rope_rates_of(r, f, 3) == nf.NF_ERR_INVALID_ARG
    assert nf.nf_rope_rates_of(None, f, 2) == nf.NF_ERR_INVALID_ARG
    assert nf.nf_rope_rates_of(r, f, -1) == nf.NF_ERR_INVALID_ARG
    for bad in (dict(dim=7), dict(dim=0), dict(dim=600), dict(dim=8, scaling="other"), dict(dim=8, frequencies=[1.0])):
        with pytest.raises(ValueError):
            nf.rope_rates(device="cpu", **bad)
    with pytest.raises(nf.NFError):
        nf.rope_rates(8, frequencies=[1.0, 2.0, 3.0, math.inf], device="cpu")


# ---------------------------------------------------------------- the entry points' checks

DIM, HQ, HK, TOKENS, BATCH = 64, 4, 2, 10, 3


def hd(data, heads=HQ, token=None, batch=None, head=DIM):
    token = heads * DIM if token is None else token
    return nf.Heads(data, TOKENS * token if batch is None else batch, token, head, heads)


def rope_arg(rates=H, dim=DIM, layout=0, magnitude=1.0, positions=I, position_bytes=8, position_stride=TOKENS):
    return nf.Rope(rates, dim, layout, magnitude, positions, position_bytes, position_stride)


def fwd(q_out=A, q=B, k_out=C, k=D, kind=nf.NF_BF16, batch=BATCH, tokens=TOKENS, dim=DIM, **kw):
    h = lambda x, n: x if x is None or isinstance(x, nf.Heads) else hd(x, n)  # noqa: E731
    rope = rope_arg(**kw)
    return nf.nf_rope_fwd(h(q_out, HQ), h(q, HQ), h(k_out, HK), h(k, HK), kind, batch, tokens, dim, rope, None)


def bwd(q_out=A, q=B, k_out=C, k=D, kind=nf.NF_BF16, batch=BATCH, tokens=TOKENS, dim=DIM, **kw):
    h = lambda x, n: x if x is None or isinstance(x, nf.Heads) else hd(x, n)  # noqa: E731
    return nf.nf_rope_bwd(h(q_out, HQ), h(q, HQ), h(k_out, HK), h(k, HK), kind, batch, tokens, dim, rope_arg(**kw), None)


def norm(q_out=A, q=B, k_out=C, k=D, kind=nf.NF_BF16, batch=BATCH, tokens=TOKENS, dim=DIM, qw=E, kw_=F, eps=1e-6, **kw):
    h = lambda x, n: x if x is None or isinstance(x, nf.Heads) else hd(x, n)  # noqa: E731
    return nf.nf_qk_rmsnorm_rope_fwd(h(q_out, HQ), h(q, HQ), qw, h(k_out, HK), h(k, HK), kw_, kind, batch, tokens, dim, eps, rope_arg(**kw), None)


def norm_grad(q_out=A, q=B, k_out=C, k=D, kind=nf.NF_BF16, batch=BATCH, tokens=TOKENS, dim=DIM, qw=E, kw_=F, eps=1e-6, dqo=G, dko=J, dqw=K,
              dkw=K + 4096, ws=L, ws_bytes=1 << 30, **kw):
    h = lambda x, n: x if x is None or isinstance(x, nf.Heads) else hd(x, n)  # noqa: E731
    return nf.nf_qk_rmsnorm_rope_bwd(h(q_out, HQ), dqw, h(dqo, HQ), h(q, HQ), qw, h(k_out, HK), dkw, h(dko, HK), h(k, HK), kw_, kind, batch,
                                     tokens, dim, eps, rope_arg(**kw), ws, ws_bytes, None)


@pytest.mark.parametrize("call", [fwd, bwd, norm, norm_grad])
def test_refusals(call):
    for dim in (0, -1, 513):
        assert call(dim=dim) == nf.NF_ERR_UNSUPPORTED_HIDDEN
    for bad in ({"kind": 2}, {"kind": -1}, {"batch": -1}, {"tokens": -1}, {"tokens": 1 << 31}, {"batch": 1 << 20, "tokens": 1 << 11},
                {"q": None}, {"q_out": None}, {"k": None}, {"k_out": None}, {"q": hd(None)}, {"q_out": hd(None)}, {"k": hd(None, HK)},
                {"q": hd(B, HQ + 1)}, {"k_out": hd(C, HQ)}, {"q": hd(B, 0)}, {"q": hd(B, token=-1)}, {"q": hd(B, batch=BIG)}, {"q": hd(B, head=-64)},
                {"rates": None}, {"positions": None}, {"dim": 32}, {"magnitude": math.nan}, {"magnitude": math.inf}, {"layout": 2},
                {"position_bytes": 2}, {"position_stride": -1},
                # outputs over inputs, over one another, or over themselves
                {"q_out": D}, {"q_out": B + 128}, {"q_out": C}, {"k_out": B + 256}, {"q_out": H}, {"q_out": I - 256}, {"k_out": I + 8},
                {"q_out": hd(A, token=0)}, {"q_out": hd(A, head=32)}, {"q_out": hd(A, batch=64)}, {"q_out": hd(B, token=512)}):
        assert call(**bad) == nf.NF_ERR_INVALID_ARG, bad
    r = rope_arg(dim=66)
    assert nf.nf_rope_fwd(hd(A), hd(B), None, None, 0, BATCH, TOKENS, DIM, r, None) == nf.NF_ERR_INVALID_ARG
    r = rope_arg(dim=7)
    assert nf.nf_rope_fwd(hd(A), hd(B), None, None, 0, BATCH, TOKENS, DIM, r, None) == nf.NF_ERR_INVALID_ARG
    for bad in ({"q": B + 1}, {"q_out": A + 1}, {"k": D + 2, "kind": nf.NF_F32}, {"rates": H + 4}, {"positions": I + 4},
                {"positions": I + 2, "position_bytes": 4}):
        assert call(**bad) == nf.NF_ERR_MISALIGNED, bad


@pytest.mark.parametrize("call", [fwd, bwd, norm, norm_grad])
def test_many_heads_are_refused(call):
    for heads in ((1 << 20) + 1, 2 ** 31 - 1):
        many = {x: nf.Heads(at, 0, 0, 64, heads) for x, at in (("q", 1 << 40), ("q_out", 2 << 40), ("dqo", 3 << 40))}
        if call is not norm_grad:
            del many["dqo"]
        assert call(batch=1, tokens=1, k=None, k_out=None, **many, **({"dko": None} if call is norm_grad else {})) == nf.NF_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [fwd, bwd, norm])
def test_nothing_to_do(call):
    assert call(tokens=0, q=hd(None), q_out=hd(None), k=hd(None, HK), k_out=hd(None, HK), rates=None, positions=None) == nf.NF_OK
    assert call(batch=0) == nf.NF_OK


def test_sets_between_one_another_are_apart():
    # the checks behind these calls end in a launch, so the last argument checked is made to fail: eps for the norm is
    # checked before, a short workspace after the overlaps (a CUDA error without a GPU)
    late = (nf.NF_ERR_WORKSPACE_TOO_SMALL, nf.NF_ERR_CUDA)
    wide = (HQ + 2 * HK) * DIM
    q, k = hd(B, HQ, token=wide), hd(B + HQ * DIM * 2, HK, token=wide)
    assert norm_grad(q_out=q, q=q, k_out=k, k=k, ws_bytes=0) in late
    # heads first: [batch, heads, tokens, dim] of the same buffer
    q = nf.Heads(B, (HQ + HK) * TOKENS * DIM, DIM, TOKENS * DIM, HQ)
    k = nf.Heads(B + HQ * TOKENS * DIM * 2, (HQ + HK) * TOKENS * DIM, DIM, TOKENS * DIM, HK)
    assert norm_grad(q_out=q, q=q, k_out=k, k=k, ws_bytes=0) in late
    # a query and a key head in turn
    q, k = nf.Heads(B, TOKENS * 512, 512, 128, 2), nf.Heads(B + 128, TOKENS * 512, 512, 128, 2)
    dq, dk = nf.Heads(G, TOKENS * 512, 512, 128, 2), nf.Heads(G + 128, TOKENS * 512, 512, 128, 2)
    assert norm_grad(q_out=q, q=q, k_out=k, k=k, dqo=dq, dko=dk, ws_bytes=0) in late
    # one element too near
    k = nf.Heads(B + 126, TOKENS * 512, 512, 128, 2)
    assert norm_grad(q_out=q, q=q, k_out=k, k=k, dqo=dq, dko=dk, ws_bytes=0) == nf.NF_ERR_INVALID_ARG
    # keys into the queries' place
    q = hd(B, HQ, token=wide)
    assert norm_grad(q_out=q, q=q, k_out=hd(B, HK, token=wide), ws_bytes=0) == nf.NF_ERR_INVALID_ARG


def test_norm_arguments():
    for call in (norm, norm_grad):
        for bad in ({"eps": 0.0}, {"eps": -1.0}, {"eps": math.nan}, {"eps": math.inf}, {"qw": None}, {"kw_": None}, {"q_out": E}, {"k_out": F - 512}):
            assert call(**bad) == nf.NF_ERR_INVALID_ARG, bad
        for bad in ({"qw": E + 1}, {"kw_": F + 2, "kind": nf.NF_F32}):
            assert call(**bad) == nf.NF_ERR_MISALIGNED, bad
    for bad in ({"dqw": None}, {"dkw": None}, {"dqo": None}, {"dko": None}, {"ws": None}, {"dkw": K + 252}, {"dqw": B}, {"dqo": hd(G, HK)},
                {"dqo": hd(None)}, {"q_out": G + 128}, {"k_out": G}):
        assert norm_grad(**bad) == nf.NF_ERR_INVALID_ARG, bad
    for bad in ({"dqw": K + 2}, {"ws": L + 2}, {"dqo": G + 1}):
        assert norm_grad(**bad) == nf.NF_ERR_MISALIGNED, bad
    for dim in (0, -1, 513):
        assert nf.nf_qk_rmsnorm_rope_bwd_workspace_size(dim) == 0


PAGES, PAGE, SEQS = 20, 16, 3


def pg(data, scale=None, page=PAGE * HK * DIM, slot=HK * DIM, head=DIM):
    return nf.Pages(data, page, slot, head, scale, PAGE * HK, HK, 1)


def append(kc=A, vc=B, cell=nf.NF_CACHE_SAME, pages=PAGES, page=PAGE, k=C, v=D, kw_=None, q_out=E, q=F, qw=None, kind=nf.NF_BF16, tokens=TOKENS,
           seqs=SEQS, dim=DIM, starts=G, past=G + 4096, table=G + 8192, stride=7, width=7, eps=1e-6, **kw):
    h = lambda x, n: x if x is None or isinstance(x, nf.Heads) else hd(x, n)  # noqa: E731
    p = lambda x, s: x if x is None or isinstance(x, nf.Pages) else pg(x, s if cell else None)  # noqa: E731
    kw = {"positions": None} | kw
    return nf.nf_kv_append(p(kc, J), p(vc, K), cell, pages, page, h(k, HK), h(v, HK), kw_, h(q_out, HQ), h(q, HQ), qw, kind, tokens, seqs, dim,
                           starts, past, table, stride, width, eps, rope_arg(**kw), None)


@pytest.mark.parametrize("cell", [nf.NF_CACHE_SAME, nf.NF_CACHE_E4M3, nf.NF_CACHE_INT8])
def test_append_refusals(cell):
    for dim in (0, -1, 513):
        assert append(cell=cell, dim=dim) == nf.NF_ERR_UNSUPPORTED_HIDDEN
    for bad in ({"kc": None}, {"vc": None}, {"k": None}, {"v": None}, {"q": None}, {"q_out": None}, {"q": None, "q_out": None, "qw": L},
                {"cell": 3}, {"cell": -1}, {"pages": -1}, {"pages": 1 << 31}, {"page": 0}, {"page": -1}, {"seqs": -1}, {"seqs": (1 << 30) + 1},
                {"width": -1}, {"stride": 6}, {"stride": -1}, {"kind": 2}, {"tokens": -1}, {"tokens": 1 << 31}, {"past": None}, {"table": None},
                {"k": hd(None, HK)}, {"v": hd(D, HQ)}, {"q_out": hd(E, HK)}, {"kc": pg(None, J)}, {"kc": pg(A, J, slot=-1)}, {"kc": pg(A, J, page=BIG)},
                {"qw": L, "eps": 0.0}, {"kw_": L, "eps": math.nan}, {"rates": None}, {"layout": 3}, {"magnitude": math.nan},
                # overlaps
                {"kc": B}, {"kc": pg(A, J, slot=32)}, {"kc": pg(A, J, page=0)}, {"kc": C}, {"vc": D}, {"kc": F}, {"vc": E + 16}, {"kc": G}, {"vc": G + 8192},
                {"q_out": C}, {"q_out": D}, {"q_out": F + 128}, {"q_out": A}, {"kc": H}, {"k": E}, {"q_out": G + 4096 - 64}, {"kw_": A + 256}, {"qw": E + 256}):
        assert append(**({"cell": cell} | bad)) == nf.NF_ERR_INVALID_ARG, bad
    for bad in ({"k": C + 1}, {"v": D + 1}, {"q": F + 1}, {"starts": G + 2}, {"past": G + 4098}, {"table": G + 8194}, {"rates": H + 4},
                {"kw_": L + 1}, {"positions": I + 4}):
        assert append(**({"cell": cell} | bad)) == nf.NF_ERR_MISALIGNED, bad
    assert append(cell=cell, tokens=0, past=None, table=None) == nf.NF_OK
    assert append(cell=cell, seqs=0, past=None, table=None) == nf.NF_OK


def test_append_scales():
    e = nf.NF_CACHE_E4M3
    for bad in ({"kc": pg(A, None)}, {"kc": pg(A, K)}, {"vc": pg(B, A + 64)}, {"kc": pg(A, C)}, {"vc": pg(B, G)}):
        assert append(cell=e, **bad) == nf.NF_ERR_INVALID_ARG, bad
    assert append(cell=e, kc=pg(A, J + 2)) == nf.NF_ERR_MISALIGNED
    assert append(kc=A + 1) == nf.NF_ERR_MISALIGNED


def test_helper_refusals():
    q, w = torch.zeros(3, 4, 64), torch.zeros(64)
    p, rates = torch.zeros(3, dtype=torch.int64), nf.rope_rates(64, device="cpu")
    for call in (lambda: nf.rope_fwd(q, None, p, rates), lambda: nf.rope_bwd(q, None, p, rates),
                 lambda: nf.qk_rmsnorm_rope_fwd(q, None, w, None, p, rates), lambda: nf.qk_rmsnorm_rope_bwd(q, None, q, None, w, None, p, rates),
                 lambda: nf.kv_append(q, q, q, q, p, p)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: nf.rope_fwd(None, None, p, rates), lambda: nf.rope_fwd(q.double(), None, p, rates),
                 lambda: nf.qk_rmsnorm_rope_bwd(q, None, None, None, w, None), lambda: nf.kv_append(None, q, q, q, p, p)):
        with pytest.raises(TypeError):
            call()


def test_binding_constants_match_the_header():
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "nf.h")).read()
    assert nf.HEAD_MAX_DIM == int(re.search(r"#define NF_HEAD_MAX_DIM (\d+)", src).group(1))
    for name in ("NF_ROPE_HALF", "NF_ROPE_INTERLEAVED", "NF_ROPE_PLAIN", "NF_ROPE_LINEAR", "NF_ROPE_NTK", "NF_ROPE_PARTS", "NF_CACHE_SAME",
                 "NF_CACHE_E4M3", "NF_CACHE_INT8"):
        assert getattr(nf, name) == int(re.search(rf"\b{name} = (\d+)", src).group(1)), name


def test_overlaps_are_never_let_through():
    # random views of one small buffer against the bytes that they cover; calls that are let through end at the short
    # workspace, so nothing is ever launched
    import random
    rng = random.Random(5)
    late = (nf.NF_ERR_WORKSPACE_TOO_SMALL, nf.NF_ERR_CUDA)
    dim, let, refused = 4, 0, 0

    def covered(base, n, strides):
        return [base + 2 * (b * strides[0] + t * strides[1] + h * strides[2] + e) for b in range(n[0]) for t in range(n[1]) for h in range(n[2])
                for e in range(dim)]
    for _ in range(4000):
        n = (rng.choice([1, 2, 3]), rng.choice([1, 2, 4]))
        views = []
        for heads in (rng.choice([1, 2, 3]), rng.choice([1, 2])):
            order = rng.sample(range(3), 3)
            sizes = (n[0], n[1], heads)
            strides, step = [0, 0, 0], dim * rng.choice([1, 1, 2, 3])
            for d in order:
                strides[d] = step
                step *= sizes[d] * rng.choice([1, 1, 2])
            if views and rng.random() < 0.7:  # the same steps as the other
                strides = views[0][2]
            views.append((sizes, A + 2 * rng.choice([0, 1, 4, 8, 12, 16, 24, 32, 48, 64, 100]), strides))
        q, k = (nf.Heads(base, *strides, sizes[2]) for sizes, base, strides in views)
        far = [nf.Heads(x << 36, 10 ** 6, 10 ** 4, 100, h) for x, h in ((2, q.heads), (3, k.heads), (4, q.heads), (5, k.heads))]
        bytes_of = [covered(base, sizes, strides) for sizes, base, strides in views]
        own = any(len(set(b)) < len(b) for b in bytes_of)
        shared = own or bool(set(bytes_of[0]) & set(bytes_of[1]))
        # both as outputs; and k as an input beside the output q
        for dk, dk_in in ((k, far[1]), (far[3], k)):
            st = nf.nf_qk_rmsnorm_rope_bwd(q, K, far[0], far[2], E, dk, K + 4096, far[1], dk_in, F, nf.NF_BF16, n[0], n[1], dim, 1e-6, None, L, 0, None)
            bad = shared if dk is k else len(set(bytes_of[0])) < len(bytes_of[0]) or bool(set(bytes_of[0]) & set(bytes_of[1]))
            assert st == nf.NF_ERR_INVALID_ARG or (st in late and not bad), (views, st)
            let += st in late
            refused += bad
    assert let > 1000 and refused > 1000
