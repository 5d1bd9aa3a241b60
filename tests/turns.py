"""2 pi to 200 bits, by Machin's formula: the reference of the rotary angles at far positions."""
from __future__ import annotations

from fractions import Fraction


def _arctan_inverse(n: int, one: int) -> int:
    """arctan(1 / n) times one, by its series."""
    term, total, k = one // n, one // n, 1
    while term:
        term //= n * n
        k += 2
        total += (-1) ** (k // 2) * (term // k)
    return total


TWO_PI = Fraction(8 * (4 * _arctan_inverse(5, 1 << 220) - _arctan_inverse(239, 1 << 220)), 1 << 220)
