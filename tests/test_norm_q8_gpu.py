"""RMSNorm with an 8-bit output against the definition in 64 bits.

Tolerances.  One fp32 rounding is u = 2^-24 relative.  The sum of squares
adds nonnegative terms in a chain of at most 16 + 1 + 5 + 32 additions (a
thread's vectors, its pair, the warp, the CTA's warps), so with the terms'
own roundings it is within 60 u; the root halves that, and the mean, eps and
rsqrt add fewer than 6 u.  y takes 3 more products, the scale 2: all of them
stay within D = 2^-18 = 64 u.  q is the nearest 8-bit value of y / scale,
whose operands are each within D: half a step, plus 2 D relative.
"""
import pytest
import torch

import row_normalization_inner_gb300 as nf
import workloads

pytestmark = pytest.mark.gpu

EPS = 1e-6
D = 2.0 ** -18
QMAX = {"e4m3": 448.0, "int8": 127.0}


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    yield


def reference(x, res, w, fmt, group):
    """(residual sums, y / scale, scale) in 64 bits."""
    s = x.double() + (0 if res is None else res.double())
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + EPS) * w.double()
    rows, hidden = y.shape
    width = group or hidden
    groups = -(-hidden // width)
    pad = torch.zeros(rows, groups * width, dtype=torch.float64, device=y.device)
    pad[:, :hidden] = y
    pad = pad.view(rows, groups, width)
    scale = (pad.abs().amax(2) / QMAX[fmt]).clamp(min=2.0 ** -100)
    v = (pad / scale[..., None]).view(rows, -1)[:, :hidden]
    return s, v, scale if group else scale[:, 0]


def check(q, scale, v, scale_ref, fmt):
    assert q.dtype == (torch.float8_e4m3fn if fmt == "e4m3" else torch.int8)
    assert scale.shape == scale_ref.shape
    assert torch.all((scale.double() - scale_ref).abs() <= D * scale_ref)
    # e4m3: half a step is 2^-4 of the value, 2^-10 below the smallest normal
    half = 0.5 if fmt == "int8" else torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10)
    assert torch.all((q.double() - v).abs() <= half + 2 * D * v.abs())


SHAPES = [(1, 8), (3, 64), (5, 120), (7, 128), (2, 136), (9, 1000), (16, 4096), (257, 1024), (259, 1032),
          (300, 5120), (260, 12288), (258, 16392), (3, 20000), (2, 32768), (257, 32768), (1, 12296)]


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,hidden", SHAPES)
def test_rmsnorm_q8(rows, hidden, fmt, group):
    x, w = workloads.rms_inputs(rows, hidden, seed=rows + hidden, device="cuda")
    keep = x.clone()
    q, scale = nf.rmsnorm_q8(x, w, EPS, fmt=fmt, group=group)
    _, v, ref = reference(x, None, w, fmt, group)
    check(q, scale, v, ref, fmt)
    assert torch.equal(x, keep)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,hidden", SHAPES)
def test_fused_add_rmsnorm_q8(rows, hidden, fmt, group):
    x, r, w = workloads.fused_inputs(rows, hidden, seed=rows + hidden, residual_scale=4.0, device="cuda")
    keep, res = x.clone(), r.clone()
    q, scale = nf.fused_add_rmsnorm_q8(x, res, w, EPS, fmt=fmt, group=group)
    s, v, ref = reference(x, r, w, fmt, group)
    check(q, scale, v, ref, fmt)
    assert torch.all((res.double() - s).abs() <= (2.0 ** -8 + 2.0 ** -23) * s.abs())
    assert torch.equal(x, keep)
    # the residual is the one the bf16 operator leaves, bit for bit
    x2, r2 = x.clone(), r.clone()
    with nf.forced_path("dynamic"):
        nf.fused_add_rmsnorm(x2, r2, w, EPS)
    assert torch.equal(res, r2)


# enough rows for every resident CTA to walk several (rows that no CTA count divides), CTAs of 128 to 1024 threads
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,hidden", [(2003, 4096), (1501, 5128), (1301, 8192), (1111, 12280), (777, 16392),
                                         (401, 32768), (3001, 3208)])
def test_many_rows(rows, hidden, fmt, group):
    x, w = workloads.rms_inputs(rows, hidden, seed=rows, device="cuda")
    x[5] = 0
    x[rows - 1, hidden - 1] = float("nan")
    keep = x.clone()
    q, scale = nf.rmsnorm_q8(x, w, EPS, fmt=fmt, group=group)
    _, v, ref = reference(x[:-1], None, w, fmt, group)
    check(q[:-1], scale[:-1], v, ref, fmt)
    assert torch.isnan(scale[-1]).all() and torch.all(bits(q[-1]) == 0)
    assert torch.all(bits(q[5]) & 0x7F == 0)
    assert torch.equal(x[:-1], keep[:-1])
    assert nf.nf_get_device_status(0) == nf.NF_OK  # no wait ran out
    # in a graph and on rows a larger buffer holds
    out, sc = torch.empty_like(q), torch.empty_like(scale)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nf.rmsnorm_q8(x, w, EPS, fmt=fmt, group=group, out=out, scale=sc)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(q)) and torch.equal(sc[:-1], scale[:-1])


def bits(q):
    return q.view(torch.uint8)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("rows", [8, 300])
def test_rows_of_zeros_nan_and_infinity(fmt, group, rows):
    hidden = 640
    x, w = workloads.rms_inputs(rows, hidden, seed=5, device="cuda")
    x[0] = 0
    x[1, 200] = float("nan")
    x[2, 639] = float("inf")
    x[3, 0] = -float("inf")
    x[4] = 3e38  # squares overflow
    x[5] = 1e-30
    q, scale = nf.rmsnorm_q8(x, w, EPS, fmt=fmt, group=group)
    assert torch.all(scale[0] == 2.0 ** -100) and torch.all(bits(q[0]) & 0x7F == 0)
    for r in (1, 2, 3, 4):
        assert torch.isnan(scale[r]).all() and torch.all(bits(q[r]) == 0), r
    _, v, ref = reference(x[5:], None, w, fmt, group)
    check(q[5:], scale[5:], v, ref, fmt)
    # a weight that is not finite reaches its own scale only
    w[130] = float("inf")
    q, scale = nf.rmsnorm_q8(x[5:], w, EPS, fmt=fmt, group=group)
    if group:
        assert not torch.isfinite(scale[:, 1]).any() and torch.all(bits(q[:, 128:256]) == 0)
        assert torch.isfinite(scale[:, [0, 2, 3, 4]]).all()
    else:
        assert not torch.isfinite(scale).any() and torch.all(bits(q) == 0)


def test_smallest_scale_holds():
    # normalized values around 2^-100 * Q: the clamped scale leaves small or zero q
    x = torch.ones(4, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.full((256,), 1.0, dtype=torch.bfloat16, device="cuda") * 2.0 ** -99
    q, scale = nf.rmsnorm_q8(x, w, EPS, fmt="int8")
    assert torch.all(scale == 2.0 ** -100) and torch.all(q == 2)


def test_leading_dimensions_outputs_and_refusals():
    x, w = workloads.rms_inputs(12, 256, seed=3, device="cuda")
    q0, s0 = nf.rmsnorm_q8(x, w, EPS, group=128)
    q1, s1 = nf.rmsnorm_q8(x.view(3, 4, 256), w, EPS, group=128)
    assert q1.shape == (3, 4, 256) and s1.shape == (3, 4, 2)
    assert torch.equal(bits(q0), bits(q1).view(12, 256)) and torch.equal(s0, s1.view(12, 2))
    out, sc = torch.empty_like(q0), torch.empty_like(s0)
    q2, s2 = nf.rmsnorm_q8(x, w, EPS, group=128, out=out, scale=sc)
    assert q2 is out and s2 is sc and torch.equal(bits(out), bits(q0)) and torch.equal(sc, s0)
    e, es = nf.rmsnorm_q8(x[:0], w, EPS)
    assert e.shape == (0, 256) and es.shape == (0,)
    with pytest.raises(ValueError):
        nf.rmsnorm_q8(x, w[:128].clone(), EPS)
    with pytest.raises(ValueError):
        nf.rmsnorm_q8(x, w, EPS, group=64)
    with pytest.raises(ValueError):
        nf.rmsnorm_q8(x, w, EPS, fmt="e5m2")
    with pytest.raises(ValueError):
        nf.rmsnorm_q8(x.t(), w, EPS)
    with pytest.raises(ValueError):
        nf.rmsnorm_q8(x, w, EPS, scale=torch.empty(3, device="cuda"))
    with pytest.raises(TypeError):
        nf.rmsnorm_q8(x, w, EPS, out=torch.empty(12, 256, dtype=torch.int8, device="cuda"))
    with pytest.raises(nf.NFError):
        nf.rmsnorm_q8(x[:, :4].contiguous(), w[:4].clone(), EPS)
    with pytest.raises(nf.NFError):
        nf.rmsnorm_q8(x, w, -1.0)


def test_another_stream_and_graph():
    x, r, w = workloads.fused_inputs(64, 2048, seed=9, device="cuda")
    want_r = r.clone()
    want = nf.fused_add_rmsnorm_q8(x, want_r, w, EPS, group=128)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r1 = r.clone()
    side.wait_stream(torch.cuda.current_stream())
    q, s = nf.fused_add_rmsnorm_q8(x, r1, w, EPS, group=128, stream=side)
    side.synchronize()
    assert torch.equal(bits(q), bits(want[0])) and torch.equal(s, want[1]) and torch.equal(r1, want_r)
    r2 = r.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, s = nf.fused_add_rmsnorm_q8(x, r2, w, EPS, group=128)
    for _ in range(3):
        r2.copy_(r)
        q.view(torch.uint8).zero_()
        graph.replay()
        assert torch.equal(bits(q), bits(want[0])) and torch.equal(s, want[1]) and torch.equal(r2, want_r)
