"""The quotient of the quantised writes (csrc/fp4.cuh, Quotient), step by step in exact arithmetic: it is the
fp32 division's for bf16 x over fp32 s, so that values on a tie of the codes stay there.  Of all 2^30 pairs of
significands the ones closest to such a tie are gone through here, and random ones."""
import random
from fractions import Fraction as F

import pytest


def rn(x):
    """x rounded to 24 bits, to the nearest, ties to even."""
    if x == 0:
        return F(0)
    m = abs(x)
    e = m.numerator.bit_length() - m.denominator.bit_length()
    if m < F(2) ** e:
        e -= 1
    unit = F(2) ** (e - 23)
    n, rest = divmod(m, unit)
    if rest * 2 > unit or (rest * 2 == unit and n % 2):
        n += 1
    return (n if x > 0 else -n) * unit


def quotient(x, s):
    r = rn(1 / s)
    q = rn(x * r)
    return rn(q - rn(q * s - x) * r)


def test_rounding():
    assert rn(F(1) + F(2) ** -24) == 1 and rn(F(1) + F(3) * F(2) ** -24) == 1 + F(2) ** -22
    assert rn(F(2) - F(2) ** -25) == 2 and rn(-F(1, 3)) == -F(11184811, 2 ** 25)


# Significands of s near multiples of 2^20, whose quotients by bf16 values come closest to the codes' ties;
# k = 16 from below only
@pytest.mark.parametrize("k", range(8, 17))
def test_next_to_ties(k):
    for d in range(-6, 7):
        S = (k << 20) + d
        if 1 << 23 <= S < 1 << 24:
            s = F(S, 1 << 23)
            for X in range(128, 256):
                x = F(X, 128)
                assert quotient(x, s) == rn(x / s), (S, X)


def test_at_random():
    r = random.Random(5)
    for _ in range(20000):
        s, x = F(r.randrange(1 << 23, 1 << 24), 1 << 23), F(r.randrange(128, 256), 128)
        assert quotient(x, s) == rn(x / s)


def test_the_remainder_is_not_always_exact():
    """The result does not rest on it."""
    r, found = random.Random(6), 0
    for _ in range(5000):
        s, x = F(r.randrange((1 << 24) - 70000, 1 << 24), 1 << 23), F(r.randrange(240, 256), 128)
        q = rn(x * rn(1 / s))
        found += rn(q * s - x) != q * s - x
    assert found
