"""The arithmetic of the 4-bit write's division, step by step in exact numbers: a quotient from a rounded
reciprocal, corrected by its exact remainder (P. Markstein, "Computation of elementary functions on the IBM
RISC System/6000 processor", 1990), is the correctly rounded one for every scale that E4M3 has."""
from fractions import Fraction

import numpy as np
import pytest


def rounded(x):
    """The fp32 number nearest to x >= 0 (a Fraction; ties to even; no denormals here)."""
    if x == 0:
        return Fraction(0)
    e = 0
    while x >= 1 << (24 + e):
        e += 1
    while x < Fraction(1 << 23) * Fraction(2) ** e:
        e -= 1
    step = Fraction(2) ** e
    return round(x / step) * step  # (round of a Fraction: ties to even)


@pytest.mark.parametrize("m", range(8, 16))
def test_reciprocal(m):
    """One step from any approximation that is off by two units in the last place or less gives the nearest
    fp32 number to 1 / s (another exponent of s changes no bit of it)."""
    s = Fraction(m, 8)
    nearest = rounded(1 / s)
    unit = Fraction(1, 1 << (23 if m == 8 else 24))
    for off in range(-2, 3):
        r = nearest + off * unit
        left = 1 - s * r
        assert left.numerator.bit_length() <= 24  # a fused multiply-add has it exactly
        assert rounded(r + r * left) == nearest


@pytest.mark.parametrize("m", range(8, 16))
def test_quotient(m):
    """For y at and around every border between codes, and many others: y r, its exact remainder, and the
    corrected quotient, against y / s."""
    s = Fraction(m, 8)
    r = rounded(1 / s)
    rng = np.random.RandomState(m)
    ys = [Fraction(int(v), 1 << 23) for v in rng.randint(1 << 23, 1 << 24, 1000)]
    for border in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        y = np.float32(border * m / 8)
        for _ in range(40):
            ys.append(Fraction(float(y)))
            y = np.nextafter(y, np.float32(100))
        y = np.float32(border * m / 8)
        for _ in range(40):
            y = np.nextafter(y, np.float32(0))
            ys.append(Fraction(float(y)))
    for y in ys:
        q = rounded(y * r)
        left = y - q * s
        assert abs(left).numerator.bit_length() <= 24
        assert rounded(q + left * r) == rounded(y / s)
