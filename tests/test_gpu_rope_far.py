"""Rotary angles at far positions and at frequencies of any size, against exact
rational arithmetic; frequencies that are refused give NaN in their pair alone."""
import math
from fractions import Fraction

import pytest
import torch

from gpu_common import need_gpu


def arctan_of_inverse(x, bits):
    """arctan(1 / x) * 2^bits from its series, less than `bits` units off."""
    term = (1 << bits) // x
    total, n, sign = term, 1, 1
    while term:
        term //= x * x
        n, sign = n + 2, -sign
        total += sign * (term // n)
    return total


# Machin: pi / 4 = 4 arctan(1 / 5) - arctan(1 / 239), to 380 bits and more
TWO_PI = Fraction(8 * (4 * arctan_of_inverse(5, 400) - arctan_of_inverse(239, 400)), 1 << 400)

FREQS = [1e-12, 2.3e-6, 1.0, 1.9999999, 2.0, 3.9, 4.0, 6.25, 1000.0, 2.0 ** 30 + 0.3, 1e15, 2.0 ** 63, 1.7 * 2.0 ** 64,
         3.1e19, 1.9 * 2.0 ** 127, 1.999 * 2.0 ** 128]


def test_pi():
    assert abs(float(TWO_PI) - 2 * math.pi) <= 2.0 ** -51


@pytest.mark.gpu
def test_any_frequency_at_far_positions():
    # an angle is 2^-31 turns off and rounded to 24 bits of half a turn (pi 2^-25 rad),
    # sincospif good to 2 ulp (2^-22): together below 2^-20
    fm = need_gpu()
    n = 2 * len(FREQS)
    freqs = torch.tensor(FREQS + [-f for f in FREQS], dtype=torch.float64, device="cuda")
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 1000003, 77, 1, 0]], dtype=torch.int32, device="cuda")
    x = torch.zeros((1, 1, pos.shape[1], 2 * n), device="cuda")
    x[..., :n] = 1.0  # (cos, sin) of every pair
    y = fm.flashmask_rope(x, None, freqs, positions=pos)[0].cpu().double()
    back = fm.flashmask_rope_bwd(x, None, freqs, positions=pos)[0].cpu().double()
    for t, p in enumerate(pos[0].tolist()):
        for i, f in enumerate(freqs.tolist()):
            a = float(Fraction(p) * Fraction(f) % TWO_PI)
            assert abs(y[0, 0, t, i] - math.cos(a)) <= 2.0 ** -20, (p, f)
            assert abs(y[0, 0, t, n + i] - math.sin(a)) <= 2.0 ** -20, (p, f)
            assert abs(back[0, 0, t, n + i] + math.sin(a)) <= 2.0 ** -20, (p, f)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [2.0 ** 129, -2.0 ** 129, 1e300, float("inf"), float("nan")])
def test_frequencies_too_large_give_nan_in_their_pair(bad):
    fm = need_gpu()
    freqs = torch.tensor([1.0, bad, 1.99 * 2.0 ** 128, 0.0], dtype=torch.float64, device="cuda")
    x = torch.ones((1, 2, 3, 8), device="cuda")
    y, _ = fm.flashmask_rope(x, None, freqs)
    assert torch.isnan(y).view(-1, 8).all(0).tolist() == torch.isnan(y).view(-1, 8).any(0).tolist() == \
        [False, True, False, False] * 2
