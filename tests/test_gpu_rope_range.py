"""The table of a rotation over the range of frequencies for which its accuracy is promised, against angles that are reduced
by whole numbers."""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

BITS = 1300  # of the numbers below, fractions of 2^BITS


def arctan_of_inverse(n):
    power = total = (1 << BITS) // n
    k, sign = 1, 1
    while power:
        power //= n * n
        k, sign = k + 2, -sign
        total += sign * (power // k)
    return total


TWO_PI = 8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))  # Machin's formula, off by less than 2^-1200


def angle(p, f):
    """p * f modulo a turn, in [-pi, pi], off by less than 2^-50."""
    num, den = f.as_integer_ratio()
    turns = (p * num << 2 * BITS) // (den * TWO_PI)  # in units of 2^-BITS
    turns = (turns + (1 << BITS - 1)) % (1 << BITS) - (1 << BITS - 1)
    return turns / (1 << BITS) * 2 * math.pi


def test_angles_of_the_reference():
    assert math.isclose(TWO_PI / (1 << BITS), 2 * math.pi, rel_tol=1e-15)
    for p, f in ((1, 1.0), (3, -0.5), (100, 0.37), (1000, 1e-4)):
        assert abs(math.remainder(p * f, 2 * math.pi) - angle(p, f)) < 1e-12


@pytest.mark.parametrize("scale", [1.0, -0.75])
@pytest.mark.parametrize("largest", [-30, 0, 20, 42, 43])
def test_frequencies_up_to_the_largest(largest, scale):
    """Off by the angle's p 2^-64 turns (below 2^-35 of a radian here) and its rounding to 2^-32 turns (2^-33 of them,
    2^-30 of a radian); by the rest's, in eighths of a turn, to 24 bits (2^-25 of pi/4); the polynomials' remainders
    (2e-9, below 2^-28), their last sum and product (2^-25 each of at most 1) and all before (a twelfth of those); the
    product with scale (2^-25): 1.3e-7 together, and an entry is promised to 2^-22 (2.4e-7) of the scale."""
    import sliding_window_attention_swa_gb300 as swa

    rng = random.Random(largest)
    n_pos = 1 << 20
    f = [rng.choice([-1, 1]) * 2.0 ** largest * rng.uniform(0.5, 1.0) for _ in range(7)] + [2.0 ** largest]
    table = swa.swa_rope_table(torch.tensor(f, dtype=torch.float64, device="cuda"), n_pos, scale)
    swa.swa_check_device_error()
    at = sorted({0, 1, 2, n_pos - 1, *(rng.randrange(n_pos) for _ in range(600))})
    got = table[at].double().cpu()
    for i, p in enumerate(at):
        for j, x in enumerate(f):
            t = angle(p, x)
            assert abs(got[i, j] - scale * math.cos(t)) <= 2.0 ** -22 * abs(scale), (p, x)
            assert abs(got[i, 8 + j] - scale * math.sin(t)) <= 2.0 ** -22 * abs(scale), (p, x)


def test_larger_frequencies_are_finite():
    """Above the range the angle is off by more, which an entry does not show otherwise."""
    import sliding_window_attention_swa_gb300 as swa

    f = torch.tensor([2.0 ** 50, 1e30, -1e300, 1.7e308, 2.0 ** 44, 1e18, -1e25, 5e-324], dtype=torch.float64, device="cuda")
    table = swa.swa_rope_table(f, 5000)
    # (each of a pair is off by 2^-22 at most)
    assert torch.isfinite(table).all() and ((table[:, :8] ** 2 + table[:, 8:] ** 2) - 1).abs().max() < 2.0 ** -20
    # position 1 at 2^44: 2^44 * 2^-107 turns
    assert abs(table[1, 4].item() - math.cos(angle(1, 2.0 ** 44))) <= 2.0 ** -22
