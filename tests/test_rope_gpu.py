"""Rotation of heads by position, and its gradient, against the definition in
64 bits (bounds: heads_reference)."""
import pytest
import torch

import row_normalization_inner_gb300 as nf
from heads_reference import TURN, close, frequencies, fused_views, gen, heads, turn

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    yield


def check(got, x, positions, freq, magnitude=1.0, layout="half", back=False):
    ref, size = turn(x, positions, freq, magnitude, layout, back)
    close(got, ref, TURN * size)


# (batch, tokens, query heads, key heads, head_dim, rotated): one token to many, odd counts, parts of a head, heads that
# are no whole vectors or whose rotated halves are not
SHAPES = [(1, 1, 1, 1, 64, 64), (1, 1, 32, 8, 128, 128), (3, 5, 6, 2, 128, 64), (2, 33, 5, 1, 80, 80), (1, 257, 3, 3, 96, 48),
          (2, 7, 4, 4, 64, 16), (1, 40, 9, 3, 256, 256), (1, 3, 2, 2, 512, 512), (1, 3, 2, 2, 504, 128), (5, 1, 7, 7, 192, 64),
          (1, 19, 3, 1, 80, 20), (1, 19, 3, 1, 72, 48), (2, 11, 2, 1, 36, 30), (1, 9, 3, 2, 7, 6), (1, 9, 3, 2, 2, 2), (1, 5, 2, 2, 8, 2),
          (1, 2000, 12, 12, 64, 64), (2, 700, 40, 8, 128, 128), (1, 3, 1, 1, 1, 0)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("batch,tokens,hq,hk,dim,rot", SHAPES)
def test_rope(batch, tokens, hq, hk, dim, rot, kind, layout):
    g = gen(tokens + dim)
    q, k = heads(g, batch, tokens, hq, dim, kind=kind), heads(g, batch, tokens, hk, dim, kind=kind)
    positions = torch.randint(0, 9000, (batch, tokens), generator=g, device="cuda")
    freq = frequencies(rot)
    rates = nf.rope_rates(rot) if rot else torch.empty(0, dtype=torch.int64, device="cuda")
    keep = q.clone(), k.clone()
    for magnitude in (1.0, 1.25):
        qo, ko = nf.rope_fwd(q, k, positions, rates, layout, magnitude)
        assert qo.shape == q.shape and ko.shape == k.shape and qo.dtype == kind
        check(qo, q, positions, freq, magnitude, layout)
        check(ko, k, positions, freq, magnitude, layout)
        dq, dk = nf.rope_bwd(q, k, positions, rates, layout, magnitude)
        check(dq, q, positions, freq, magnitude, layout, back=True)
        check(dk, k, positions, freq, magnitude, layout, back=True)
    assert torch.equal(q, keep[0]) and torch.equal(k, keep[1])
    if rot < dim:  # the rest of a head is passed on bit for bit
        assert torch.equal(qo[..., rot:], q[..., rot:]) and torch.equal(dk[..., rot:], k[..., rot:])


# enough rows that a warp takes several, in tokens of one share, of some and of many; the last rows of a share missing or not
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("batch,tokens,hq,hk,dim,rot", [(3, 3337, 1, 0, 64, 64), (1, 10007, 3, 1, 128, 64), (2, 2503, 9, 7, 96, 96), (1, 4001, 24, 8, 80, 80),
                                                        (1, 1201, 72, 8, 128, 128), (5, 601, 33, 1, 256, 256), (1, 3001, 17, 1, 64, 32), (1, 5003, 8, 2, 128, 128),
                                                        (2, 2001, 2, 1, 80, 80), (1, 4003, 16, 5, 64, 64), (3, 1111, 4, 1, 192, 64), (1, 2999, 7, 3, 112, 112)])
def test_many_rows(batch, tokens, hq, hk, dim, rot, kind, layout):
    g = gen(tokens + dim)
    q = heads(g, batch, tokens, hq, dim, kind=kind)
    k = heads(g, batch, tokens, hk, dim, kind=kind) if hk else None
    positions, freq = torch.randint(0, 9000, (batch, tokens), generator=g, device="cuda"), frequencies(rot)
    qo, ko = nf.rope_fwd(q, k, positions, nf.rope_rates(rot), layout)
    check(qo, q, positions, freq, layout=layout)
    if hk:
        check(ko, k, positions, freq, layout=layout)
        wq, wk = nf.rope_fwd(q, k, positions, nf.rope_rates(rot), layout, q_out=q, k_out=k)
        assert torch.equal(wq, qo) and torch.equal(wk, ko)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_is_the_transpose(layout):
    # <R x, y> = <x, R^T y>, and against differences of the forward pass
    g = gen(1)
    x, y = heads(g, 1, 6, 3, 80, kind=F32), heads(g, 1, 6, 3, 80, kind=F32)
    positions, rates = torch.arange(6, device="cuda") * 37, nf.rope_rates(48)
    rx = nf.rope_fwd(x, None, positions, rates, layout, 1.1)[0].double()
    ry = nf.rope_bwd(y, None, positions, rates, layout, 1.1)[0].double()
    sizes = 4 * 1.1 * (x.abs().amax() * y.abs().amax()).double() * x.numel() * TURN
    assert abs((rx * y.double()).sum() - (x.double() * ry).sum()) <= sizes
    d = heads(g, 1, 6, 3, 80, kind=F32)
    both = nf.rope_fwd(x + d, None, positions, rates, layout, 1.1)[0].double() - rx
    size = turn((x.abs() + d.abs()), positions[None], frequencies(48), 1.1, layout)[1]
    assert torch.all((both - turn(d, positions[None], frequencies(48), 1.1, layout)[0]).abs() <= 4 * TURN * size)


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
def test_positions(ids):
    # far, negative, shared by the batch, expanded, and behind a stride
    g = gen(2)
    q = heads(g, 3, 50, 4, 128, kind=F32)
    freq, rates = frequencies(128), nf.rope_rates(128)
    far = torch.randint(-2 ** 31, 2 ** 31 - 1, (3, 50), generator=g, device="cuda").to(ids)
    # the rates are off by 2^-65 turns per position and the reference's angles by 2^-53 of theirs
    ref, size = turn(q, far, freq)
    close(nf.rope_fwd(q, None, far, rates)[0], ref, (TURN + 2.0 ** 31 * 2.0 ** -51) * size)
    one = torch.randint(0, 70000, (50,), generator=g, device="cuda").to(ids)
    want = nf.rope_fwd(q, None, one, rates)[0]
    check(want, q, one[None], freq)
    assert torch.equal(nf.rope_fwd(q, None, one.expand(3, 50), rates)[0], want)
    wide = torch.zeros(3, 64, dtype=ids, device="cuda")
    wide[:, :50] = one
    assert torch.equal(nf.rope_fwd(q, None, wide[:, :50], rates)[0], want)
    with pytest.raises(ValueError):
        nf.rope_fwd(q, None, wide[:, :49], rates)
    with pytest.raises(ValueError):
        nf.rope_fwd(q, None, torch.zeros(3, 100, dtype=ids, device="cuda")[:, ::2], rates)


def test_beyond_32_bits():
    # positions of 64 bits: the angle is exact for the rate as it is rounded
    q = torch.zeros(1, 3, 1, 8, dtype=F32, device="cuda")
    q[..., 0] = 1.0
    rates = torch.tensor([1 << 62, 1 << 30, 1, 0], dtype=torch.int64, device="cuda")  # a quarter turn, 2^-34, 2^-64, none
    positions = torch.tensor([[1, (1 << 40) + 3, -(1 << 40)]], device="cuda")
    y = nf.rope_fwd(q, None, positions, rates)[0][0, :, 0]
    assert torch.equal(y[0, [0, 4]].cpu(), torch.tensor([0.0, 1.0]))
    assert torch.equal(y[1, [0, 4]].cpu(), torch.tensor([0.0, -1.0]))
    assert torch.equal(y[2, [0, 4]].cpu(), torch.tensor([1.0, 0.0]))


def strided(x, order):
    """The same heads in another order of memory, with room between."""
    b, t, h, d = x.shape
    if order == "heads first":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if order == "tokens first":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    extra = 8 if order == "padded" else 3
    wide = torch.full((b, t + 1, h + 2, d + extra), 77.0, dtype=x.dtype, device=x.device)
    wide[:, :t, 1:h + 1, extra - 3 if order == "odd" else 0:][..., :d] = x
    return wide[:, :t, 1:h + 1, extra - 3 if order == "odd" else 0:][..., :d]


@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("dim", [128, 80, 20])
@pytest.mark.parametrize("order", ["heads first", "tokens first", "padded", "odd"])
def test_orders_and_strides(order, dim, kind):
    g = gen(3)
    q, k = heads(g, 2, 21, 5, dim, kind=kind), heads(g, 2, 21, 3, dim, kind=kind)
    positions, rates = torch.arange(21, device="cuda"), nf.rope_rates(dim // 4 * 2)
    want = nf.rope_fwd(q, k, positions, rates, "interleaved")
    got = nf.rope_fwd(strided(q, order), strided(k, order), positions, rates, "interleaved")
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = strided(torch.zeros_like(q), order)
    around = out._base.clone() if out._base is not None else None
    assert nf.rope_fwd(q, None, positions, rates, "interleaved", q_out=out)[0] is out
    assert torch.equal(out, want[0])
    if order in ("padded", "odd"):  # what lies between the heads is left as it was
        base = out._base.clone()
        out.copy_(torch.zeros_like(q))
        assert torch.equal(out._base, around) and not torch.equal(base, around)


def test_in_place_views_of_a_projection():
    g = gen(4)
    whole, (q, k, v) = fused_views(g, 2, 37, [8, 2, 2], 128, BF)
    keep, positions, rates = whole.clone(), torch.arange(37, device="cuda"), nf.rope_rates(128)
    want = nf.rope_fwd(q, k, positions, rates)
    got = nf.rope_fwd(q, k, positions, rates, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, keep[:, :, 10:])
    nf.rope_bwd(q, k, positions, rates, dq=q, dk=k)  # and back: two roundings to bf16 in all
    assert torch.all((q.float() - keep[:, :, :8].float()).abs() <= 2.0 ** -6 * keep[:, :, :8].float().abs().amax())
    # k's turned heads into q's place, or a part of an input
    with pytest.raises(nf.NFError):
        nf.rope_fwd(q[:, :, :2], k, positions, rates, k_out=q[:, :, 1:3])
    with pytest.raises(nf.NFError):
        nf.rope_fwd(q[:, 1:], None, positions[1:], rates, q_out=q[:, :-1])
    with pytest.raises(nf.NFError):  # rows that coincide
        nf.rope_fwd(q, None, positions, rates, q_out=torch.empty(2, 1, 8, 128, dtype=BF, device="cuda").expand(2, 37, 8, 128))
    # heads that all queries share are read as often as they are there
    one = heads(g, 2, 37, 1, 128)
    got = nf.rope_fwd(one.expand(2, 37, 8, 128), None, positions, rates)[0]
    assert torch.equal(got, nf.rope_fwd(one, None, positions, rates)[0].expand(2, 37, 8, 128))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot", [(128, 64), (80, 20), (96, 96)])
def test_infinities_and_nan_stay_in_their_pairs(dim, rot, layout):
    g = gen(5)
    x = heads(g, 1, 9, 3, dim, kind=F32)
    positions, rates = 1 + torch.arange(9, device="cuda"), nf.rope_rates(rot)
    want = nf.rope_fwd(x, None, positions, rates, layout)[0]
    for value in (float("inf"), float("nan")):
        for i in (1, rot - 1, dim - 1):
            y = x.clone()
            y[0, 4, 1, i] = value
            got = nf.rope_fwd(y, None, positions, rates, layout)[0]
            changed = torch.zeros_like(want, dtype=torch.bool)
            a, b = (i % (rot // 2), i % (rot // 2) + rot // 2) if layout == "half" else (i & ~1, i | 1)
            for e in ((a, b) if i < rot else (i, i)):
                changed[0, 4, 1, e] = True
            assert torch.equal(got[~changed], want[~changed])
            assert not torch.isfinite(got[changed]).any()


def test_scalings_reach_the_angles():
    g = gen(6)
    q = heads(g, 1, 64, 2, 64, kind=F32)
    positions = torch.randint(0, 100000, (1, 64), generator=g, device="cuda")
    f = frequencies(64)
    for scaling, ref in (("plain", f), ("linear", f / 8), ("ntk", frequencies(64, 10000.0 * 8 ** (64 / 62)))):
        rates = nf.rope_rates(64, scaling=scaling, factor=8.0)
        check(nf.rope_fwd(q, None, positions, rates)[0], q, positions, ref)
    rates = nf.rope_rates(64, frequencies=-f)
    check(nf.rope_fwd(q, None, positions, rates)[0], q, positions, f, back=True)


def test_empty_streams_and_graphs():
    g = gen(7)
    rates = nf.rope_rates(128)
    for shape in ((0, 5, 4, 128), (2, 0, 4, 128)):
        q = torch.empty(shape, dtype=BF, device="cuda")
        out, none = nf.rope_fwd(q, None, torch.empty(shape[:2], dtype=torch.int64, device="cuda"), rates)
        assert out.shape == shape and none is None
    q, k = heads(g, 64, 1, 32, 128), heads(g, 64, 1, 8, 128)
    positions = torch.randint(0, 4000, (64, 1), generator=g, device="cuda")
    want = nf.rope_fwd(q, k, positions, rates)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = nf.rope_fwd(q, k, positions, rates, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = nf.rope_fwd(q, k, positions, rates)
    for shift in (0, 5):
        positions += shift
        want = nf.rope_fwd(q, k, positions, rates)
        graph.replay()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals():
    q = torch.zeros(2, 3, 4, 64, dtype=BF, device="cuda")
    p, rates = torch.zeros(2, 3, dtype=torch.int64, device="cuda"), nf.rope_rates(64)
    bad = [(TypeError, dict(q=q.half())), (TypeError, dict(k=q.float())), (TypeError, dict(rates=rates.int())), (TypeError, dict(rates=None)),
           (TypeError, dict(positions=p.float())), (ValueError, dict(positions=None)), (ValueError, dict(positions=p[:1])),
           (ValueError, dict(layout="other")), (ValueError, dict(q=q[0, 0])), (ValueError, dict(k=q[:1])), (ValueError, dict(k=q[..., :32])),
           (ValueError, dict(q=q.transpose(2, 3))), (ValueError, dict(rates=nf.rope_rates(66))), (ValueError, dict(q_out=q[:, :, :2])),
           (TypeError, dict(q_out=q.float())), (ValueError, dict(k=None, k_out=q)), (ValueError, dict(q=q.cpu(), k=None)),
           (ValueError, dict(rates=rates.cpu())), (nf.NFError, dict(magnitude=float("nan"))), (nf.NFError, dict(q=q[:, :, :0], k=None)),
           (nf.NFError, dict(q_out=q.clone().as_strided(q.shape, (768, 256, 32, 1))))]
    for error, change in bad:
        kw = dict(q=q, k=q, positions=p, rates=rates) | change
        with pytest.raises(error):
            nf.rope_fwd(**kw)
    big = torch.zeros(1, 1, 1, 520, dtype=BF, device="cuda")
    with pytest.raises(nf.NFError):
        nf.rope_fwd(big, None, p[:1, :1], rates)


def test_strides_of_single_dimensions_do_not_count():
    # one head, one token or one batch whose stride is no whole vector: the same bits as from contiguous rows
    g = gen(8)
    rates = nf.rope_rates(64)
    for shape, strides in (((3, 7, 1, 64), (7 * 64, 64, 13, 1)), ((5, 1, 4, 64), (256, 3, 64, 1)), ((1, 9, 2, 64), (5, 128, 64, 1))):
        x = heads(g, *shape)
        odd = torch.zeros(2000 * 8, dtype=BF, device="cuda").as_strided(shape, strides)
        odd.copy_(x)
        p = torch.arange(shape[1], device="cuda")
        assert torch.equal(nf.rope_fwd(odd, None, p, rates)[0], nf.rope_fwd(x, None, p, rates)[0])
