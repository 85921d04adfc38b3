"""RMSNorm of query and key heads with the rotation in the same pass, and its
gradient, against the definition in 64 bits (bounds: heads_reference)."""
import pytest
import torch

import row_normalization_inner_gb300 as nf
from heads_reference import (NORM, TURN, close, frequencies, fused_views, gen, heads, norm_turn_grad, normed, rates_of, turn)

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    yield


def weight(g, dim, kind):
    return (1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(kind)


def check(got, x, w, eps, positions, freq, magnitude=1.0, layout="half"):
    n = normed(x, w, eps)
    ref, size = turn(n, positions, freq, magnitude, layout) if freq is not None else (n, n.abs())
    close(got, ref, (NORM + TURN) * size)


SHAPES = [(1, 1, 1, 1, 64, 64), (16, 1, 32, 8, 128, 128), (3, 5, 6, 2, 128, 64), (2, 33, 5, 1, 80, 80), (1, 257, 3, 3, 96, 48),
          (1, 40, 9, 3, 256, 256), (1, 3, 2, 2, 512, 512), (1, 19, 3, 1, 80, 20), (2, 11, 2, 1, 36, 30), (1, 9, 3, 2, 7, 6),
          (1, 5, 2, 2, 8, 2), (1, 5, 2, 2, 8, 0), (1, 7, 3, 2, 1, 0), (2, 50, 4, 2, 64, 0), (1, 1500, 12, 12, 64, 64), (2, 700, 40, 8, 128, 128), (1, 10007, 3, 1, 128, 64),
          (2, 2503, 9, 7, 96, 96), (1, 1201, 72, 8, 128, 128), (5, 601, 33, 1, 256, 256), (1, 3001, 17, 1, 64, 0), (1, 5003, 8, 2, 128, 128), (2, 2001, 2, 1, 80, 80), (3, 1111, 16, 3, 64, 64)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("batch,tokens,hq,hk,dim,rot", SHAPES)
def test_forward_and_gradient(batch, tokens, hq, hk, dim, rot, kind, layout):
    g = gen(tokens + dim)
    q, k = heads(g, batch, tokens, hq, dim, kind=kind, scale=3.0), heads(g, batch, tokens, hk, dim, kind=kind)
    qw, kw = weight(g, dim, kind), weight(g, dim, kind)
    positions = torch.randint(0, 9000, (batch, tokens), generator=g, device="cuda") if rot else None
    freq, magnitude = (frequencies(rot), 1.25) if rot else (None, 1.0)
    kept = [t.clone() for t in (q, k, qw, kw)]
    qo, ko = nf.qk_rmsnorm_rope_fwd(q, k, qw, kw, positions, rates_of(rot), EPS, layout, magnitude)
    check(qo, q, qw, EPS, positions, freq, magnitude, layout)
    check(ko, k, kw, EPS, positions, freq, magnitude, layout)
    dqo, dko = heads(g, batch, tokens, hq, dim, kind=kind), heads(g, batch, tokens, hk, dim, kind=kind)
    args = (dqo, dko, q, k, qw, kw, positions, rates_of(rot), EPS, layout, magnitude)
    got = nf.qk_rmsnorm_rope_bwd(*args)
    for dx, dw, dy, x, w in ((got[0], got[2], dqo, q, qw), (got[1], got[3], dko, k, kw)):
        assert dx.shape == x.shape and dx.dtype == kind and dw.shape == (dim,) and dw.dtype == F32
        rdx, rdw, off_dx, off_dw = norm_turn_grad(dy, x, w, EPS, positions, freq, magnitude, layout)
        close(dx, rdx, off_dx)
        close(dw, rdw, off_dw)
    assert all(torch.equal(a, b) for a, b in zip(kept, (q, k, qw, kw)))
    # every sum has a fixed order
    assert all(torch.equal(a, b) for a, b in zip(got, nf.qk_rmsnorm_rope_bwd(*args)))
    # one kind of heads alone
    check(nf.qk_rmsnorm_rope_fwd(q, None, qw, None, positions, rates_of(rot), EPS, layout, magnitude)[0], q, qw, EPS, positions, freq, magnitude, layout)
    alone = nf.qk_rmsnorm_rope_bwd(dko, None, k, None, kw, None, positions, rates_of(rot), EPS, layout, magnitude)
    assert alone[1] is None and alone[3] is None
    assert torch.equal(alone[0], got[1])
    _, rdw, _, off_dw = norm_turn_grad(dko, k, kw, EPS, positions, freq, magnitude, layout)
    close(alone[2], rdw, off_dw)


def test_gradient_against_differences():
    # d sum(c y) / d x and / d w in the direction of a small step, 64-bit forms of both sides
    g = gen(11)
    x, w, c = heads(g, 1, 3, 2, 48, kind=F32), weight(g, 48, F32), heads(g, 1, 3, 2, 48, kind=F32)
    p, freq = torch.tensor([[5, 9, 100]], device="cuda"), frequencies(32)
    dx, _, dw, _ = nf.qk_rmsnorm_rope_bwd(c, None, x, None, w, None, p, rates_of(32), EPS)
    u, v = torch.randn_like(x).double(), torch.randn_like(w).double()

    def loss(t):
        return (c.double() * turn(normed(x.double() + t * u, w.double() + t * v, EPS), p, freq)[0]).sum()
    h = 1e-4
    slope = (loss(h) - loss(-h)) / (2 * h)
    got = (dx.double() * u).sum() + (dw.double() * v).sum()
    # the third derivative's share is h^2 / 6 of a value of the slope's own order; the kernel's fp32 below 2^-15
    sizes = (dx.double() * u).abs().sum() + (dw.double() * v).abs().sum()
    assert abs(got - slope) <= (2.0 ** -15 + 1e3 * h * h) * sizes


def test_many_rows_and_orders():
    # several rows to every warp of every CTA, from a projection's views into other orders
    g = gen(12)
    for kind, dim, hq, hk in ((BF, 128, 24, 4), (F32, 80, 10, 10), (BF, 20, 16, 5)):
        whole, (q, k, v) = fused_views(g, 3, 1301, [hq, hk, hk], dim, kind)
        keep = whole.clone()
        qw, kw = weight(g, dim, kind), weight(g, dim, kind)
        positions, rot = torch.arange(1301, device="cuda"), dim // 4 * 2
        freq, rates = frequencies(rot), rates_of(rot)
        dqo = heads(g, 3, hq, 1301, dim, kind=kind).transpose(1, 2)
        dko = heads(g, 3, hk, 1301, dim, kind=kind).transpose(1, 2)
        dwhole = torch.zeros_like(whole)
        dq, dk, dv = torch.split(dwhole, [hq, hk, hk], 2)
        got = nf.qk_rmsnorm_rope_bwd(dqo, dko, q, k, qw, kw, positions, rates, EPS, dq=dq, dk=dk)
        assert got[0] is dq and got[1] is dk and not dv.any() and torch.equal(whole, keep)
        for dx, dw, dy, x, w in ((dq, got[2], dqo, q, qw), (dk, got[3], dko, k, kw)):
            rdx, rdw, off_dx, off_dw = norm_turn_grad(dy, x, w, EPS, positions[None], freq)
            close(dx, rdx, off_dx)
            close(dw, rdw, off_dw)
        # the gradient in the place of the output's gradient, or of the input
        want = dq.clone(), dk.clone()
        a, b = dqo.clone(), dko.clone()
        nf.qk_rmsnorm_rope_bwd(a, b, q, k, qw, kw, positions, rates, EPS, dq=a, dk=b)
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
        nf.qk_rmsnorm_rope_bwd(dqo, dko, q, k, qw, kw, positions, rates, EPS, dq=q, dk=k)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, keep[:, :, hq + hk:])
        # forward, in place
        whole.copy_(keep)
        want = nf.qk_rmsnorm_rope_fwd(q, k, qw, kw, positions, rates, EPS)
        nf.qk_rmsnorm_rope_fwd(q, k, qw, kw, positions, rates, EPS, q_out=q, k_out=k)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, keep[:, :, hq + hk:])


@pytest.mark.parametrize("kind", [BF, F32])
def test_rows_of_zeros_nan_and_infinity(kind):
    g = gen(13)
    x, dy, w = heads(g, 1, 40, 4, 128, kind=kind), heads(g, 1, 40, 4, 128, kind=kind), weight(g, 128, kind)
    p, rates = torch.arange(40, device="cuda"), rates_of(128)
    want, dwant = nf.qk_rmsnorm_rope_fwd(x, None, w, None, p, rates)[0], nf.qk_rmsnorm_rope_bwd(dy, None, x, None, w, None, p, rates)[0]
    x[0, 0] = 0
    x[0, 1, 2, 7] = float("nan")
    x[0, 2, 3, 100] = float("inf")
    x[0, 3] = 3e38
    got = nf.qk_rmsnorm_rope_fwd(x, None, w, None, p, rates)[0]
    assert torch.all(got[0, 0] == 0) and torch.isnan(got[0, 1, 2]).all() and torch.isnan(got[0, 2, 3]).any()
    assert torch.all(got[0, 3] == 0)  # the sum of squares is infinite
    assert torch.equal(got[0, 4:], want[0, 4:]) and torch.equal(got[0, 1, [0, 1, 3]], want[0, 1, [0, 1, 3]])
    dx = nf.qk_rmsnorm_rope_bwd(dy, None, x, None, w, None, p, rates)[0]
    assert torch.equal(dx[0, 4:], dwant[0, 4:]) and torch.equal(dx[0, 1, [0, 1, 3]], dwant[0, 1, [0, 1, 3]])
    rdx, _, off, _ = norm_turn_grad(dy[:, :1], x[:, :1], w, EPS, p[None, :1], frequencies(128))
    close(dx[:, :1], rdx, off)
    assert torch.isnan(dx[0, 1, 2]).all()


def test_empty_workspace_streams_and_graphs():
    g = gen(14)
    w, rates = weight(g, 64, BF), rates_of(64)
    e = torch.empty(2, 0, 3, 64, dtype=BF, device="cuda")
    p = torch.empty(2, 0, dtype=torch.int64, device="cuda")
    assert nf.qk_rmsnorm_rope_fwd(e, e, w, w, p, rates)[0].shape == e.shape
    got = nf.qk_rmsnorm_rope_bwd(e, e, e, e, w, w, p, rates)
    assert got[0].shape == e.shape and not got[2].any() and not got[3].any()
    q, k = heads(g, 4, 100, 8, 64), heads(g, 4, 100, 2, 64)
    dq, dk, p = heads(g, 4, 100, 8, 64), heads(g, 4, 100, 2, 64), torch.arange(100, device="cuda")
    args = (dq, dk, q, k, w, w, p, rates)
    want = nf.qk_rmsnorm_rope_bwd(*args)
    size = nf.nf_qk_rmsnorm_rope_bwd_workspace_size(64)
    ws = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")  # its contents do not matter, what lies behind is left
    got = nf.qk_rmsnorm_rope_bwd(*args, workspace=ws[:size])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.all(ws[size:] == 255)
    with pytest.raises(nf.NFError):
        nf.qk_rmsnorm_rope_bwd(*args, workspace=ws[:size - 1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = nf.qk_rmsnorm_rope_bwd(*args, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd = nf.qk_rmsnorm_rope_fwd(q, k, w, w, p, rates)
        got = nf.qk_rmsnorm_rope_bwd(*args)
    for _ in range(3):
        q.mul_(1.5)
        want = nf.qk_rmsnorm_rope_bwd(*args)
        fwant = nf.qk_rmsnorm_rope_fwd(q, k, w, w, p, rates)
        for t in got + fwd:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got + fwd, want + fwant))


def test_refusals():
    g = gen(15)
    q, w, rates = heads(g, 2, 3, 4, 64), weight(g, 64, BF), rates_of(64)
    p = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
    bad = [(TypeError, dict(q_weight=None)), (TypeError, dict(q_weight=w.float())), (ValueError, dict(q_weight=w[:32])),
           (TypeError, dict(k_weight=None)), (ValueError, dict(k=None)), (nf.NFError, dict(eps=0.0)), (nf.NFError, dict(eps=float("nan"))),
           (ValueError, dict(rates=None)), (ValueError, dict(positions=None)), (nf.NFError, dict(q_out=q[:, :, :1].expand(2, 3, 4, 64))),
           (ValueError, dict(layout=None))]
    for error, change in bad:
        kw = dict(q=q, k=q, q_weight=w, k_weight=w, positions=p, rates=rates) | change
        with pytest.raises(error):
            nf.qk_rmsnorm_rope_fwd(**kw)
    d = heads(g, 2, 3, 4, 64)
    bad = [(ValueError, dict(dq_out=d[:, :, :2])), (TypeError, dict(dk_out=None)), (TypeError, dict(dq_out=d.float())),
           (ValueError, dict(dk=d[:, :2])), (nf.NFError, dict(dq=d, dk=d)), (nf.NFError, dict(dq=q[:, :, :].flip(0) * 0 + 0, eps=-1.0)),
           (ValueError, dict(k=None, dk_out=None, k_weight=None, dk=d))]
    for error, change in bad:
        kw = dict(dq_out=d, dk_out=d.clone(), q=q, k=q.clone(), q_weight=w, k_weight=w, positions=p, rates=rates) | change
        with pytest.raises(error):
            nf.qk_rmsnorm_rope_bwd(**kw)


@pytest.mark.parametrize("dim", [64, 200, 63, 400])
@pytest.mark.parametrize("kind", [nf.NF_BF16, nf.NF_F32])
def test_gradient_without_rows_reads_nothing(kind, dim):
    # null pointers for all that has no rows, the weights too: the weights' gradients are zeros
    n = nf.nf_qk_rmsnorm_rope_bwd_workspace_size(dim)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dw = torch.full((2, dim), 7.0, device="cuda")
    q, k = nf.Heads(None, 0, 6 * dim, dim, 4), nf.Heads(None, 0, 6 * dim, dim, 2)
    for sets in (1, 2):
        dw.fill_(7.0)
        two = (lambda x: x) if sets == 2 else (lambda x: None)
        assert nf.nf_qk_rmsnorm_rope_bwd(q, dw[0].data_ptr(), q, q, None, two(k), two(dw[1].data_ptr()), two(k), two(k), None, kind, 2, 0,
                                         dim, 1e-6, None, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == nf.NF_OK
        assert not dw[:sets].any() and (dw[sets:] == 7.0).all()
