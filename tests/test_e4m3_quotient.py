"""The quotient step of the row operators' E4M3 encoder (fg_e4m3_quot.hpp):
q = x * inv, then one correction by the exact residual. It can leave the correctly
rounded quotient only where x / s lies within 2^-23 ulp of the middle of two floats,
and the code can then change only if one of the two is a boundary between E4M3 codes
(at most 5 significant bits). Every such pair of significands is checked here in exact
arithmetic, and random ones besides."""
import random
from fractions import Fraction as F

import numpy as np


def rounded(v):
    """v to 24 significant bits, ties to even, no limits on the exponent."""
    if v == 0:
        return F(0)
    sign, v, e = (1 if v > 0 else -1), abs(v), 0
    while v >= 2 ** 24:
        v, e = v / 2, e + 1
    while v < 2 ** 23:
        v, e = v * 2, e - 1
    n = int(v)
    r = v - n
    if r > F(1, 2) or (r == F(1, 2) and n & 1):
        n += 1
    return sign * F(n) * F(2) ** e


def corrected(x, s, inv):
    q = rounded(x * inv)
    return rounded(q - rounded(q * s - x) * inv)


def near_pairs():
    """(S, X), 24-bit significands with X / S within 2^-20 ulp of a float midpoint beside a code boundary: 2 X of the
    right power of two is S (2 m +- 1) to within 8, with m a multiple of 2^19, so S is within 8 of a multiple of 2^20."""
    for c in range(8, 16):
        for d in range(-8, 9):
            S = c * 2 ** 20 + d
            if not 2 ** 23 <= S < 2 ** 24:
                continue
            for m5 in range(1, 32):
                m = m5
                while m < 2 ** 23:
                    m *= 2
                mids = [F(2 * m + 1, 2), F(2 * m - 1, 2)] + ([F(4 * m - 1, 4)] if m == 2 ** 23 else [])
                for mid in mids:
                    for e in (23, 24, 25):
                        x0 = int(mid * S / F(2) ** e)
                        for X in range(x0 - 2, x0 + 4):
                            if 2 ** 23 <= X < 2 ** 24 and abs(F(X) * F(2) ** e / S - mid) <= F(1, 2 ** 20):
                                yield S, X


def test_every_pair_beside_a_code_boundary():
    n = 0
    for S, X in near_pairs():
        n += 1
        assert corrected(F(X), F(S), rounded(F(1, S))) == rounded(F(X, S)), (S, X)
    assert n > 200


def test_random_pairs():
    rng = random.Random(1)
    for _ in range(2000):
        S, X = rng.randrange(2 ** 23, 2 ** 24), rng.randrange(2 ** 23, 2 ** 24)
        q = corrected(F(X), F(S), rounded(F(1, S)))
        assert q == rounded(F(X, S))


def test_every_pair_just_below_a_power_of_two():
    """The band that near_pairs leaves out: S within 8 below 2^24, the neighbours of 16 x 2^20."""
    n = 0
    for S in range(2 ** 24 - 8, 2 ** 24):
        for m5 in range(16, 32):
            m = m5 * 2 ** 19
            for mid in [F(2 * m + 1, 2), F(2 * m - 1, 2)] + ([F(4 * m - 1, 4)] if m == 2 ** 23 else []):
                for e in (23, 24, 25):
                    x0 = int(mid * S / F(2) ** e)
                    for X in range(x0 - 2, x0 + 4):
                        if 2 ** 23 <= X < 2 ** 24 and abs(F(X) * F(2) ** e / S - mid) <= F(1, 2 ** 20):
                            n += 1
                            assert corrected(F(X), F(S), rounded(F(1, S))) == rounded(F(X, S)), (S, X)
    assert n > 20


def test_quotients_pass_448_by_one_float_at_most():
    """Every significand of amax: amax / (amax / 448), both rounded, is 448 or a neighbour, which is why the encoder's
    quotients need no clamp; no value of a block is above its amax."""
    a = np.arange(2 ** 23, 2 ** 24, dtype=np.int64).astype(np.float32)
    q = a / (a / np.float32(448))
    below, above = (np.nextafter(np.float32(448), np.float32(to)) for to in (0, 1000))
    assert set(np.unique(q).tolist()) == {float(below), 448.0, float(above)}
