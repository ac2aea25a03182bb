"""A rotation's turns a position, as append has them: f / 2 pi behind the point, to the last of 64 bits."""
import ctypes
import random
from fractions import Fraction

import pytest


@pytest.fixture(scope="module")
def capi():
    from mhc_residual_boundary_gb300 import build
    build.build()
    from mhc_residual_boundary_gb300 import capi as c
    c.lib()
    return c


def two_pi():
    """To 2^-250, by Machin's formula: pi / 4 = 4 arctan(1 / 5) - arctan(1 / 239)."""
    one = 1 << 300

    def arctan(x):
        term, total, n, sign = one // x, 0, 1, 1
        while term:
            total += sign * (term // n)
            term //= x * x
            n, sign = n + 2, -sign
        return total
    return Fraction(8 * (4 * arctan(5) - arctan(239)), one)


def frequencies():
    rng = random.Random(7)
    out = [0.0, -0.0, 1.0, -1.0, 3.141592653589793, 6.283185307179586, -6.283185307179586, 1000.0, 12345678.9, 1e-9, -1e-9,
           5e-324, 1e-300, -1e-25, 2.0 ** 40 - 2.0 ** -13, -(2.0 ** 39)]
    out += [theta ** (-2.0 * i / r) for theta, r in ((10000.0, 64), (500000.0, 128), (1e6, 128)) for i in range(r // 2)]
    out += [rng.choice((-1, 1)) * 2.0 ** rng.uniform(-80, 40) for _ in range(2000)]
    return out


def test_turns(capi):
    full = two_pi()
    for f in frequencies():
        want = Fraction(f) / full % 1 * 2 ** 64
        got = capi.mhc_test_attention_turns(f)
        off = abs(got - want)
        assert min(off, 2 ** 64 - off) <= 1, f


def test_frequencies_of_2_40_and_more_are_refused(capi):
    for f in (2.0 ** 40, -2.0 ** 40, 1e300, float("inf"), float("nan")):
        values = (ctypes.c_double * 8)(*[1.0] * 7, f)
        with pytest.raises(capi.MhcError, match="INVALID_ARG"):
            capi.mhc_attention_create(capi.mhc_attention_config_t(16, 4, 128, 64, 16, 0, 1.0, values), 0)
    with pytest.raises(capi.MhcError, match="frequency 1 "):   # 2^0, then 2^42 by a theta below one
        capi.mhc_attention_create(capi.mhc_attention_config_t(16, 4, 128, 64, 32, 0, 2.0 ** -336 * 2.0 ** -336, None), 0)
