"""The 64-bit fractions of a turn are the integers next to the formula's numbers, so that position times
fraction is off by at most 2^31 / 2 of 2^-64 of a turn, 2^-34, at any position.

The formula's numbers are powers of rational ones: with E the exact fraction times 2^64 and d the dimension,
E^(d/2) = (2^64 / 2 pi)^(d/2) / base^i, so the integer T is the nearest one if (T - 1/2)^(d/2) <= that <=
(T + 1/2)^(d/2); pi to 70 digits (Machin's formula, whole numbers) leaves no doubt."""
import math
from decimal import Decimal
from fractions import Fraction

import pytest

from trellis_decode_gemv_gb300 import binding as B


def pi():
    one = 10 ** 80

    def arctan(n):                                     # arctan(1 / n) * 10^80
        total = term = one // n
        k, sign = 3, -1
        while term:
            term //= n * n
            total += sign * (term // k)
            k, sign = k + 2, -sign
        return total
    return Fraction(4 * (4 * arctan(5) - arctan(239)), one)


TURN = Fraction(2 ** 64) / (2 * pi())


def fractions(f):
    return [t % 2 ** 64 for t in f.freqs.tolist()]


def nearest(got, powered, power):
    """Whether `got` is the integer next to the `power`-th root of `powered`."""
    return (Fraction(2 * got - 1, 2)) ** power <= powered <= (Fraction(2 * got + 1, 2)) ** power


@pytest.mark.parametrize("dim", [16, 64, 96, 128])
@pytest.mark.parametrize("base", [10000, 500000, 1000000])
@pytest.mark.parametrize("scaling,scale", [("none", 1), ("linear", 3.5)])
def test_powers_of_the_base(dim, base, scaling, scale):
    f = fractions(B.exl3_rotary_freqs(dim, base=float(base), scaling=scaling, scale=float(scale), device="cpu"))
    for i, t in enumerate(f):
        assert nearest(t, (TURN / Fraction(scale)) ** (dim // 2) / Fraction(base) ** i, dim // 2), i


@pytest.mark.parametrize("dim,scale", [(16, 8), (32, 4)])
def test_a_larger_base(dim, scale):
    f = fractions(B.exl3_rotary_freqs(dim, base=10000.0, scaling="ntk", scale=float(scale), device="cpu"))
    for i, t in enumerate(f):                          # base^(-2i/d) scale^(-2i/(d-2))
        power = dim * (dim - 2) // 2
        assert nearest(t, TURN ** power / Fraction(10000) ** (i * (dim - 2)) / Fraction(scale) ** (i * dim), power), i


@pytest.mark.parametrize("scaling,scale", [("llama3", 8), ("yarn", 32)])
def test_pairs_that_stay_and_pairs_that_are_scaled(scaling, scale):
    """The fastest are as they are, the slowest over scale (what lies between mixes both: held to 2^-48 elsewhere)."""
    dim, base = 128, 500000
    f = fractions(B.exl3_rotary_freqs(dim, base=float(base), scaling=scaling, scale=float(scale), original=4096, device="cpu"))
    for i, over in ((0, 1), (1, 1), (10, 1), (dim // 2 - 1, scale), (dim // 2 - 2, scale)):
        assert nearest(f[i], (TURN / over) ** (dim // 2) / Fraction(base) ** i, dim // 2), i


def test_radians_of_their_own():
    given = [1.0, 0.1, 1 / 3, 1e-7, 6.2, Fraction(1, 3), Decimal("0.1"), 0.0, -0.5]
    f = fractions(B.Exl3RotaryFreqs(given, device="cpu"))
    assert f == [round(Fraction(r) * TURN) % 2 ** 64 for r in given]
    for bad in (math.nan, math.inf):
        with pytest.raises((ValueError, OverflowError)):
            B.Exl3RotaryFreqs([bad], device="cpu")


def test_numbers_of_other_types():
    np = pytest.importorskip("numpy")
    want = fractions(B.exl3_rotary_freqs(64, base=10000.0, scaling="llama3", scale=8.0, original=8192, device="cpu"))
    assert fractions(B.exl3_rotary_freqs(64, base=10000, scaling="llama3", scale=np.float32(8), original=np.int64(8192), device="cpu")) == want
    assert fractions(B.Exl3RotaryFreqs(np.array([1.0, 0.25], np.float32), device="cpu")) == fractions(B.Exl3RotaryFreqs([1.0, 0.25], device="cpu"))
