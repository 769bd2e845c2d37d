"""Frequencies of any size become turns (no GPU)."""
from fractions import Fraction

import pytest


def half_turn(digits):
    """pi by Euler's arctan formula for 1/2 and 1/3, in decimals: another way than the library's."""
    one = 10 ** (digits + 10)

    def arctan_inverse(n):
        total = term = one * n // (n * n + 1)
        k = 1
        while term:
            term = term * 2 * k // ((2 * k + 1) * (n * n + 1))
            total += term
            k += 1
        return total

    return Fraction(4 * (arctan_inverse(2) + arctan_inverse(3)), one)


@pytest.mark.parametrize("f", [1.0, 1e-4, -0.7, 2.0 ** 60 + 2.0 ** 10, 2.0 ** 100, -1e30, 1e300, 1.7976931348623157e308,
                               5e-324, 2.0 ** -70, 0.0])
def test_turns_of_any_frequency(f):
    """To the last bit of 64, against pi to 500 digits: 2^1024 takes 309 of them before the point."""
    from serial_draft_head_gb300 import tree
    want = Fraction(f) / (2 * half_turn(500)) % 1 * 2 ** 64
    off = abs(tree._turns(f) - want)
    assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 2 ** 40), f


def test_frequencies_that_are_no_numbers_are_refused():
    import torch
    from serial_draft_head_gb300 import Rotation
    for bad in (float("inf"), float("nan")):
        with pytest.raises(ValueError):
            Rotation(32, torch.full((16,), bad, dtype=torch.float64), device="cuda:0")
