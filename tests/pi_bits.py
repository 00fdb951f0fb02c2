"""Pi as a fraction, from Machin's formula in whole numbers."""
from fractions import Fraction
from functools import lru_cache


@lru_cache(None)
def two_pi(bits: int) -> Fraction:
    """2 pi, off by less than 2^-bits."""
    one = 1 << (bits + 32)

    def arctan_of_one_over(x):
        term, total, n = one // x, 0, 1
        while term:
            total += term // n if n % 4 == 1 else -(term // n)
            term //= x * x
            n += 2
        return total

    return Fraction(2 * (16 * arctan_of_one_over(5) - 4 * arctan_of_one_over(239)), one)
