"""The reciprocals of the 4-bit cache's writer. Its quotients are correctly rounded if they go
through a correctly rounded reciprocal (Markstein); the scale's is refined from an approximation
within one unit in the last place, y0 + (1 - s y0) y0 in two fused multiply-adds, and for every
fp16 scale that gives the correctly rounded one whatever the approximation is. The range's
division by 15 goes through RN(1 / 15) in the same way."""
from fractions import Fraction

import numpy as np


def rn(x):
    """Fraction to the nearest fp32 (ties to even), as a Fraction; normal range only."""
    if x == 0:
        return x
    sign = -1 if x < 0 else 1
    x = abs(x)
    e = x.numerator.bit_length() - x.denominator.bit_length()
    e -= 1 if x < Fraction(2) ** e else 0
    unit = Fraction(2) ** (e - 23)
    n, rest = divmod(x, unit)
    if rest * 2 > unit or (rest * 2 == unit and n % 2):
        n += 1
    return sign * n * unit


def fma(a, b, c):
    return rn(a * b + c)


def test_reciprocal_of_every_significand():
    for m in range(1024, 2048):              # the exponent only shifts all values
        s = Fraction(m, 1024)
        y = rn(1 / s)
        ulp = Fraction(2) ** -24 if y < 1 else Fraction(2) ** -23
        for k in (-1, 0, 1):
            y0 = y + k * ulp
            assert fma(fma(-s, y0, Fraction(1)), y0, y0) == y, (m, k)


def test_division_by_fifteen():
    r = rn(Fraction(1, 15))
    rng = np.random.default_rng(0)
    for a in np.concatenate([np.arange(1, 4096, dtype=np.float32), rng.random(4096, np.float32),
                             np.abs(rng.standard_normal(4096)).astype(np.float32) * np.float32(1000)]):
        a = Fraction(float(a))
        q0 = rn(a * r)
        assert fma(fma(-q0, Fraction(15), a), r, q0) == rn(a / 15)
