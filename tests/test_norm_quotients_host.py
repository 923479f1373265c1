"""The norm's two quotients, written out in FP32 as its kernel has them, against exact rational arithmetic: the scale
amax / 448 is the nearest FP32 number, 448 / most is b + bl to 2^-44 from any reciprocal within 2^-23 (the bound of the
hardware's).  An FMA of FP32 numbers is one rounding of the exact value."""

from fractions import Fraction

import numpy as np
import pytest

F = np.float32


def rounded(v: Fraction) -> Fraction:
    """Nearest FP32 number, ties to even (no overflow, no subnormals here)."""
    if v == 0:
        return v
    sign, v = (-1, -v) if v < 0 else (1, v)
    e = v.numerator.bit_length() - v.denominator.bit_length()
    if Fraction(2) ** e > v:
        e -= 1
    step = Fraction(2) ** (e - 23)
    return sign * round(v / step) * step  # (Python rounds halves to even)


def mul(a, b):
    return rounded(a * b)


def fma(a, b, c):
    return rounded(a * b + c)


def numbers(n, lo, hi, seed):
    """FP32 numbers over the binades lo .. hi, the ends of each among them."""
    rng = np.random.default_rng(seed)
    v = np.ldexp(1 + rng.random(n), rng.integers(lo, hi, n)).astype(F)
    edges = [F(np.ldexp(m, e)) for e in range(lo, hi, 7) for m in (1.0, 1.0 + 2.0 ** -23, 2.0 - 2.0 ** -23, 1.75)]
    return [Fraction(float(x)) for x in np.concatenate([v, np.array(edges, dtype=F)])]


def test_rounding_is_fp32s():
    rng = np.random.default_rng(0)
    for x in rng.standard_normal(2000) * 10.0 ** rng.integers(-20, 20, 2000):
        assert rounded(Fraction(float(x))) == Fraction(float(F(x)))


def test_the_scale_is_the_nearest_quotient():
    inv = Fraction(float(F(1) / F(448)))
    for amax in numbers(20000, -99, 99, 1):
        s = mul(amax, inv)
        got = fma(fma(Fraction(-448), s, amax), inv, s)
        assert got == rounded(amax / 448)


@pytest.mark.parametrize("off", [Fraction(0), Fraction(1, 2 ** 23), -Fraction(1, 2 ** 23), Fraction(1, 2 ** 24)])
def test_the_double_quotient(off):
    worst = Fraction(0)
    for most in numbers(5000, -59, 99, 2):
        r = rounded((1 + off) / most)  # (up to 2^-22.4 off)
        b = mul(Fraction(448), r)
        bl = mul(fma(-b, most, Fraction(448)), r)
        worst = max(worst, abs((b + bl) * most / 448 - 1))
    assert worst < Fraction(1, 2 ** 44)
