"""Angles of far positions in exact arithmetic (test infrastructure): pi as a fraction
from Machin's formula, 320 bits."""
from fractions import Fraction


def _arctan_inverse(n, bits):
    """arctan(1 / n) in units of 2^-bits."""
    term = total = (1 << bits) // n
    k, sign = 1, 1
    while term:
        term //= n * n
        k += 2
        sign = -sign
        total += sign * (term // k)
    return total


PI = Fraction(4 * (4 * _arctan_inverse(5, 336) - _arctan_inverse(239, 336)), 1 << 336)


def turns(w, p=1):
    """The fraction of a turn of p * w radians, in [0, 1); w is a double, taken exactly."""
    x = Fraction(w) * p / (2 * PI)
    return x - (x.numerator // x.denominator)
