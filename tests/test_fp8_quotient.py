"""The quantiser's quotient is the IEEE one for every pair of bf16 significands, in exact arithmetic.

A block's scale is s = m / 448 rounded to 24 bits, m its largest magnitude, and a value's quotient x / s is formed as
r = 1 / s, q = x r, q - (q s - x) r, each step rounded to 24 bits.  Powers of two change nothing as long as no step
leaves the normal numbers, so the significands of m and x, 8 bits each, are all there is."""
from __future__ import annotations

from fractions import Fraction


def rounded(v: Fraction) -> Fraction:
    """To 24 bits, to nearest, ties to even."""
    if v == 0:
        return v
    size, sign = abs(v), -1 if v < 0 else 1
    e = size.numerator.bit_length() - size.denominator.bit_length()
    if Fraction(2) ** e > size:
        e -= 1
    unit = Fraction(2) ** (e - 23)
    n, rest = divmod(size, unit)
    n += rest * 2 > unit or (rest * 2 == unit and n & 1)
    return sign * n * unit


def test_every_pair_of_significands():
    inexact = 0
    for m in range(128, 256):
        s = rounded(Fraction(m, 448))
        r = rounded(1 / s)
        for x in range(128, 256):
            q = rounded(x * r)
            left = rounded(q * s - x)
            inexact += left != q * s - x
            assert rounded(q - left * r) == rounded(x / s), (m, x)
    assert inexact == 35
