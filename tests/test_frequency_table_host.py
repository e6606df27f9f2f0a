"""How far the entries of pa_rotary_frequencies are from the frequencies themselves, in 60 decimal digits.

An entry theta / (2 pi), theta = base^(-2 i / R), is off, in units of 2^-53 of itself, by: the exponent's rounding, times
|ln theta|; pow, 2 (an ulp); a division by the factor or a mix of two products and a sum, 4; the constant 2 pi and the
division by it, 2; and, where the base is changed, the exponent R / (R - 2) and its pow, 4, times 2 i / R <= 1.  theta
(12 + |ln theta|) <= 12 for theta <= 1, so 12 / (2 pi) < 2 units at the most: 2^-52 of a turn, as include/pa.h states."""
from decimal import Decimal, getcontext

import pytest

import paged_decode_attention_reshape_gb300 as pa

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_decode_attention_reshape_gb300 import _build
    _build.build()
    pa.lib()


def turns(R, base, scaling, factor, L0, low, high):
    base, factor = Decimal(base), Decimal(factor)
    if scaling == pa.PA_ROTARY_BASE:
        base *= (factor.ln() * R / (R - 2)).exp()
    out = []
    for i in range(R // 2):
        theta = (base.ln() * (-2 * i) / R).exp()
        if scaling == pa.PA_ROTARY_LINEAR:
            theta /= factor
        if scaling == pa.PA_ROTARY_PARTS:
            n = L0 * theta / (2 * PI)
            keep = min(Decimal(1), max(Decimal(0), (n - low) / (high - low)))
            theta = keep * theta + (1 - keep) * theta / factor
        out.append(theta / (2 * PI))
    return out


@pytest.mark.parametrize("R", [2, 16, 48, 64, 80, 96, 112, 128, 176, 256])
@pytest.mark.parametrize("base", [1.0, 3.7, 10000.0, 150000.0, 500000.0, 1e8])
@pytest.mark.parametrize("scaling,factor", [(pa.PA_ROTARY_PLAIN, 1.0), (pa.PA_ROTARY_LINEAR, 3.3), (pa.PA_ROTARY_BASE, 8.0),
                                            (pa.PA_ROTARY_PARTS, 32.0)])
def test_entries(R, base, scaling, factor):
    if scaling == pa.PA_ROTARY_BASE and R == 2:
        return
    got = pa.pa_rotary_frequencies(R, base, scaling, factor, 4096.0, 1.0, 32.0).tolist()
    for f, want in zip(got, turns(R, base, scaling, factor, 4096, 1, 32)):
        assert abs(Decimal(f % 2 ** 64) / 2 ** 64 - want) <= Decimal(2) ** -52
