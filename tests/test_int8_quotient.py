"""The integer quantisers divide in three fp32 steps: inv = 1 / s, q = x inv, q' = q - (q s - x) inv.
q' may differ from the rounded quotient only where x / s is within 2^-23 ulp of the middle of two floats,
and its nearest integer only where one of the two is half an integer. Every pair of significands that
close to such a middle (with a margin of four) is gone through here in exact arithmetic."""
from fractions import Fraction


def rn(v):
    """v (a Fraction) to the nearest float of 24 bits, ties to even, without limits of the exponent."""
    if v == 0:
        return v
    n, e = abs(v), 0
    while n >= 2 ** 24:
        n, e = n / 2, e + 1
    while n < 2 ** 23:
        n, e = n * 2, e - 1
    k, rest = divmod(n.numerator, n.denominator)
    twice = 2 * rest
    if twice > n.denominator or (twice == n.denominator and k % 2):
        k += 1
    return (1 if v > 0 else -1) * Fraction(k) * Fraction(2) ** e


def nearest(v):
    """The nearest integer, ties to even."""
    return round(v)


def by_steps(x, s):
    inv = rn(1 / s)
    q = rn(x * inv)
    return rn(q - rn(q * s - x) * inv)


def middles():
    """(M, k): M / 2^k is the middle of half an integer up to 126.5 and a float beside it."""
    for H in range(1, 254, 2):
        k = 25 - H.bit_length()          # H 2^k has 25 bits: its last one is half an ulp of H / 2
        yield H * 2 ** k + 1, k + 1
        if H == 1:                       # 0.5: the floats below it are twice as close
            yield H * 2 ** (k + 1) - 1, k + 2
        else:
            yield H * 2 ** k - 1, k + 1


def pairs():
    """(s, x): significands S, X of 24 bits with |X 2^B - S M| <= 8, i.e. x / s within 2^-21 ulp of the middle."""
    for M, k in middles():
        for B in (23, 24, 25, 26):
            inverse = pow(M, -1, 2 ** B)
            for D in range(-8, 9):
                S = D * inverse % 2 ** B
                while S < 2 ** 24:
                    if S >= 2 ** 23:
                        X, rest = divmod(S * M - D, 2 ** B)
                        assert rest == 0
                        if 2 ** 23 <= X < 2 ** 24:
                            yield Fraction(S), Fraction(X) * Fraction(2) ** B / 2 ** k
                    S += 2 ** B


def test_codes_are_those_of_the_rounded_quotient():
    n = 0
    for s, x in pairs():
        assert nearest(by_steps(x, s)) == nearest(rn(x / s)), (s, x)
        n += 1
    assert n > 1000


def test_pairs_are_where_they_should_be():
    for i, (s, x) in enumerate(pairs()):
        if i % 50 == 0:
            v = x / s
            near_half = min(abs(v - Fraction(h, 2)) for h in range(1, 254, 2))
            assert near_half < Fraction(1, 2 ** 16)


def test_the_largest_quotient_rounds_to_127():
    """The row's largest value over its own scale, whatever its significand: s = rn(a / 127)."""
    import numpy as np
    a = (np.arange(2 ** 23, 2 ** 24, dtype=np.int64)).astype(np.float32)
    s = a / np.float32(127)
    assert np.all(np.rint(a / s) == 127)
