"""Angles of rotary positions without rounding, for the tests: pi to 300 bits
and rational arithmetic."""
from fractions import Fraction
import math


def _arccot(x, one):
    total = term = one // x
    n, sign = 3, -1
    while term:
        term //= x * x
        total += sign * (term // n)
        sign, n = -sign, n + 2
    return total


_ONE = 1 << 320
# Machin: pi / 4 = 4 arccot 5 - arccot 239
PI = Fraction(4 * (4 * _arccot(5, _ONE) - _arccot(239, _ONE)), _ONE)


def turns(freq):
    """freq radians in turns."""
    return Fraction(freq) / (2 * PI)


def cos_sin(pos, freq):
    """cos and sin of pos * freq, the angle reduced to [-1/2, 1/2] turns exactly."""
    t = int(pos) * turns(freq)
    angle = float((t - round(t)) * 2 * PI)
    return math.cos(angle), math.sin(angle)
