"""The rates of a rotation against 60 decimal digits (no GPU needed).

A rate is the nearest multiple of 2^-64 to its share of a turn.  The host
computes in pairs of doubles, some 104 bits; 2^-80 of a frequency below 1 would
be 2^-16 of a rate's unit.  A rate therefore is within 1/2 + 2^-10 units of the
exact share, whatever machine made it.
"""
import math
from decimal import Decimal, getcontext

import pytest

import row_normalization_inner_gb300 as nf

TWO_PI = Decimal("6.2831853071795864769252867665590057683943387987502116419498891846")
UNITS = Decimal(2) ** 64


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    getcontext().prec = 60
    yield


def off(rates, frequencies):
    """The largest distance in units of 2^-64, modulo a turn."""
    worst = Decimal(0)
    for r, f in zip(rates.tolist(), frequencies):
        d = (Decimal(r) - f / TWO_PI * UNITS) % UNITS
        worst = max(worst, min(abs(d), UNITS - abs(d)))
    return worst


NEAR = Decimal("0.501")


def plain(dim, base):
    step = -2 * Decimal(base).ln() / dim
    return [(i * step).exp() for i in range(dim // 2)]


@pytest.mark.parametrize("base", [10000.0, 1e6, 500000.0, 1.0000001, 3.7, 1e300, 10000.1])
@pytest.mark.parametrize("dim", [2, 20, 64, 128, 512])
def test_plain_and_linear(dim, base):
    f = plain(dim, base)
    assert off(nf.rope_rates(dim, base, device="cpu"), f) <= NEAR
    for factor in (1.0, 8.0, 3.3):
        assert off(nf.rope_rates(dim, base, scaling="linear", factor=factor, device="cpu"), [x / Decimal(factor) for x in f]) <= NEAR


@pytest.mark.parametrize("factor", [1.0, 8.0, 40.0, 1.7])
@pytest.mark.parametrize("dim", [4, 64, 128])
def test_ntk_and_parts(dim, factor):
    s = Decimal(factor)
    longer = (Decimal(10000).ln() + s.ln() * dim / (dim - 2)) * -2 / dim
    assert off(nf.rope_rates(dim, scaling="ntk", factor=factor, device="cpu"), [(i * longer).exp() for i in range(dim // 2)]) <= NEAR
    for length, low, high in ((8192.0, 1.0, 32.0), (4096.0, 0.3, 4.7), (100.0, 0.0, 1e-3)):
        want = []
        for x in plain(dim, 10000.0):
            keep = (Decimal(length) * x / TWO_PI - Decimal(low)) / (Decimal(high) - Decimal(low))
            keep = min(max(keep, Decimal(0)), Decimal(1))
            want.append(x * (keep + (1 - keep) / s))
        assert off(nf.rope_rates(dim, scaling="parts", factor=factor, length=length, low=low, high=high, device="cpu"), want) <= NEAR


def test_given_frequencies():
    f = [1.0, -1.0, 2 * math.pi, 0.1, 1e-9, 1000.0, 1e-300, -1e-4, 1048575.9, -1048575.1, 3.0, 0.0, 1e-19, 2.0 ** -60, 6.283185307179586, 0.5]
    got = nf.rope_rates(2 * len(f), frequencies=f, device="cpu")
    assert off(got, [Decimal(x) for x in f]) <= NEAR
    assert got[11] == 0 and got[6] == 0


def test_far_positions():
    # an angle at position p is off by p times what its rate is off: 2^-32 of a turn at the first 2^32 positions
    f, p = plain(128, 10000.0), 2 ** 32 - 1
    for r, x in zip(nf.rope_rates(128, device="cpu").tolist(), f):
        turns = Decimal(r * p % 2 ** 64) / UNITS - x * p / TWO_PI
        turns = turns - turns.to_integral_value()
        assert abs(turns) <= Decimal(2) ** -32
