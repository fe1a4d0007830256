"""The 4-bit cache writer's division of a group's range by 15, q0 = RN(a r) with r = RN(1 / 15) and
RN(q0 + RN(a - 15 q0) r), over every fp32 significand: the correctly rounded quotient. (The
exponent only shifts all values, as long as nothing leaves the normal range; a range below it gives the least scale.)"""
import numpy as np


def test_every_significand():
    r = np.float64(np.float32(1.0 / 15.0))
    for first in range(1 << 23, 1 << 24, 1 << 21):
        m = np.arange(first, first + (1 << 21), dtype=np.int64)
        a = m.astype(np.float64)                                  # an integer below 2^24
        q0 = (a * r).astype(np.float32).astype(np.float64)        # 48 bits: the product is exact in 64
        rest = a - 15.0 * q0                                      # 28 bits and a shared exponent: exact
        assert np.array_equal(rest, rest.astype(np.float32))      # and its rounding to fp32 changes nothing
        # RN(q0 + rest r): the product is exact, the sum's error is kept for a sum halfway between two fp32
        p = rest * r
        s = q0 + p
        bb = s - q0
        err = (q0 - (s - bb)) + (p - bb)
        q = s.astype(np.float32)
        ulp = np.spacing(np.abs(q)).astype(np.float64)
        half = np.abs(s - q.astype(np.float64)) == ulp / 2
        assert not np.any(half & (err != 0))                      # no sum is rounded twice
        # correctly rounded: 15 q is within 15 half units of a (15 is odd: never both at once)
        k = np.rint(q.astype(np.float64) / ulp).astype(np.int64)
        unit = np.rint(ulp * 2.0 ** 8).astype(np.int64)
        assert np.all(np.abs(15 * k * unit - (m << 8)) * 2 <= 15 * unit)
