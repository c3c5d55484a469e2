"""The rotation's angles to their last bits: sines near zero, and frequencies below it.

Queries (1, 0): the rotated pair is factor (cos, sin), so each output shows its own error.  Of the value: sine
and cosine 2 ulp, two products and the factor, below 2^-20; the output's rounding, 2^-11 and at least 2^-25.
In radians: the frequency in 64-bit fixed point is off by less than two units, 2^-63 of a turn a position; the
angle is rounded to fp32, 2^-24 of itself."""
import math
from fractions import Fraction

import pytest
import torch

from test_append import Tokens

TWO_PI = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)
POSITIONS = [0, 1, 2, 3, 5, -1, -3, 17, 100, 1000, 4095, 65535, 10 ** 6, -10 ** 6, 2 ** 24 + 1, 2 ** 30 + 7,
             2 ** 31 - 1, -2 ** 31]


def check(freqs, factor, inter):
    t = Tokens(torch, "f16", 1, 1, 2 * len(freqs), 2 * len(freqs), inter, [len(POSITIONS)], [0], norm=False,
               freqs=freqs, factor=factor)
    p = torch.arange(len(freqs), device="cuda")
    i, j = (2 * p, 2 * p + 1) if inter else (p, p + len(freqs))
    q = torch.zeros_like(t.q.contiguous())
    q[..., i] = 1.0
    out = torch.zeros_like(q)
    pos = torch.tensor(POSITIONS, dtype=torch.int32, device="cuda")
    t.run(t.pool.clone(), out, q=q, pos=pos)
    rows = []
    for z in POSITIONS:
        angles = [Fraction(z) * Fraction(f) % TWO_PI for f in freqs]
        rows.append([float(a if 2 * a <= TWO_PI else a - TWO_PI) for a in angles])
    angles = torch.tensor(rows, dtype=torch.float64, device="cuda")
    off = pos.double().abs()[:, None] * 2.0 ** -63 * 2 * math.pi + angles.abs() * 2.0 ** -24
    for at, want in ((i, torch.cos(angles)), (j, torch.sin(angles))):
        want = want * factor
        tol = want.abs() * (2.0 ** -20 + 2.0 ** -11) + off * abs(factor) + 2.0 ** -25
        worst = ((out[:, 0][:, at].double() - want).abs() / tol).max().item()
        assert worst <= 1, f"{worst:.3g} of the tolerance"


def geometric(n, base, stretch=1.0):
    return [base ** (-p / n) / stretch for p in range(n)]


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("factor", [1.0, 4096.0, -8192.0])
def test_sines_near_zero(inter, factor):
    check(geometric(64, 500000.0, 8.0), factor, inter)
    check(geometric(16, 1e7), factor, inter)



@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("factor", [1.0, 4096.0])
def test_frequencies_below_zero(inter, factor):
    """As exact as those above it, however small."""
    check([-f for f in geometric(64, 500000.0, 8.0)], factor, inter)
    check([f if p % 2 else -f for p, f in enumerate(geometric(16, 1e6))], factor, inter)
    check([-1e-12, -3.0, -1e-13, 5e8, -5e8, 2.0 ** 30, -0.0, -3e-14], factor, inter)
