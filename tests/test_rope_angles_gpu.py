"""The sine and cosine of an angle, each against its own value.

A pair (1, 0) turned by t comes out as (cos t, sin t): what the kernels multiply
by.  An angle is the 64-bit product of a rate and a position, a share of a turn;
its quarter is taken off exactly, and the rest x, at most 1/8 of a turn either
way, made to fp32 in two halves.  u = 2^-24 is half a step of fp32, relative.

x is within 1.5 u (where its upper half just passes 24 bits; 1.25 u from 2^-5 of
a quarter on).  The sine takes that, the last rounding (u) and those of the term
behind the first, which is at most 0.11 of it: below 2.7 u of its value.  The cosine,
at least 0.707: half a step at the end (0.5 u of 1), x^2's error of 3.5 u times
t^2 / 2 <= 0.309 and that term's own rounding (0.31 u): below 2.7 u of its value.
What the series leave out is below 0.07 u.  3 u is
allowed, of the sine and cosine themselves however small: a slow pair a few
positions on turns by 1e-6, and an element that is the other's sine alone has
no larger one beside it.
"""
import math

import pytest
import torch

import row_normalization_inner_gb300 as nf
from heads_reference import gen, rates_of

pytestmark = pytest.mark.gpu

F32 = torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    yield


def turns(rates, positions):
    """(cos, sin) in 64 bits of each position's angles, [positions, rates]."""
    angle = positions.long()[:, None] * rates[None]  # modulo 2^64, as a signed number
    quarter = ((angle >> 61) + 1) >> 1
    rest = angle - (quarter << 62)
    t = rest.double() * (2.0 ** -62 * math.pi / 2)
    c, s, q = torch.cos(t), torch.sin(t), quarter & 3
    cos = torch.where(q == 0, c, torch.where(q == 1, -s, torch.where(q == 2, -c, s)))
    sin = torch.where(q == 0, s, torch.where(q == 1, c, torch.where(q == 2, -s, -c)))
    return cos, sin


# rates from 2^-64 of a turn a position to the fastest, and those of contexts from the shortest to the longest
def rates_in_hand(g, pairs):
    log = torch.rand(pairs, generator=g, device="cuda") * 62
    return [torch.exp2(log.double()).long(), torch.randint(-2 ** 63, 2 ** 63 - 1, (pairs,), generator=g, device="cuda"), rates_of(2 * pairs),
            rates_of(2 * pairs, base=1e7, scaling="linear", factor=8.0)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,offset", [(128, 0), (72, 0), (128, 1), (18, 0)])  # lanes with both vectors, others, and element by element
def test_sines_and_cosines(dim, offset, layout):
    g, pairs = gen(dim + offset), dim // 2
    positions = torch.cat([torch.arange(200, device="cuda"), torch.randint(0, 2 ** 17, (700,), generator=g, device="cuda"),
                           torch.randint(-2 ** 62, 2 ** 62, (300,), generator=g, device="cuda")])
    first = torch.zeros(dim, device="cuda")
    a = torch.arange(pairs, device="cuda") * (1 if layout == "half" else 2)
    b = a + (pairs if layout == "half" else 1)
    first[a] = 1.0
    x = torch.zeros(len(positions) * dim + 8, device="cuda")[offset:][:len(positions) * dim].view(len(positions), 1, dim)
    x.copy_(first)
    for rates in rates_in_hand(g, pairs):
        cos, sin = turns(rates, positions)
        for back in (False, True):
            y = (nf.rope_bwd if back else nf.rope_fwd)(x, None, positions, rates, layout)[0][:, 0].double()
            for got, ref in ((y[:, a], cos), (y[:, b], -sin if back else sin)):
                bad = (got - ref).abs() > 3 * U * ref.abs()
                assert not bad.any(), (int(bad.sum()), got[bad][:4], ref[bad][:4])


@pytest.mark.parametrize("cell", [torch.float32, torch.float8_e4m3fn])
def test_slow_pairs_of_an_append(cell):
    # the keys (0, 1) of the first positions: their first elements are minus the sine alone
    dim, tokens = 128, 40
    rates = rates_of(dim, base=1e6, scaling="linear", factor=8.0)
    k = torch.zeros(tokens, 1, dim, device="cuda")
    k[..., 64:] = 1.0
    cache, scale = torch.zeros(2, 1, tokens, 1, dim, device="cuda").to(cell), torch.zeros(2, 1, tokens, 1, device="cuda")
    scales = dict(k_scale=scale[0], v_scale=scale[1]) if cell != F32 else {}
    table, past = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    q = nf.kv_append(k, k, cache[0], cache[1], table, past, starts, rates, q=k, **scales)
    cos, sin = turns(rates, torch.arange(tokens, device="cuda"))
    for got in (q[:, 0],) + ((cache[0][0, :, 0],) if cell == F32 else ()):
        for part, ref in ((got[:, :64].double(), -sin), (got[:, 64:].double(), cos)):
            assert torch.all((part - ref).abs() <= 3 * U * ref.abs())


def test_slow_pairs_of_the_gradient():
    # of rows whose norm's gradient is the row itself turned back: x at right angles to it, and of mean square 1 - eps
    dim, tokens, eps = 128, 64, 2.0 ** -20
    rates = rates_of(dim, base=1e6, scaling="linear", factor=8.0)
    positions = torch.arange(tokens, device="cuda")
    dy, w = torch.zeros(tokens, 1, dim, device="cuda"), torch.ones(dim, device="cuda")
    dy[..., :32] = 1.0
    x = torch.zeros(tokens, 1, dim, device="cuda")
    x[..., 32:64] = 2.0  # the other pairs' first elements: nothing of dy turns there
    dx = nf.qk_rmsnorm_rope_bwd(dy, None, x, None, w, None, positions, rates, eps)[0][:, 0].double()
    rstd = (1 / torch.tensor(1.0 + eps, dtype=torch.float64)).sqrt()
    cos, sin = turns(rates[:32], positions)
    # 3 u as above, rsqrt within 4 u and one product
    assert torch.all((dx[:, :32] - rstd * cos).abs() <= 9 * U * cos.abs())
    assert torch.all((dx[:, 64:96] + rstd * sin).abs() <= 9 * U * sin.abs())
