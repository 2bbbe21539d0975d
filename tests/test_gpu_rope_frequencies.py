"""Rotation by frequencies of any size, against phases from whole-number arithmetic.

Bound, elementwise: that of the other rotation tests, 32 u r with u = 2^-24 and r the length of
the rotated pair (no norm here, fp32: the rotation alone), and the angle's own error as stated,
|position| (2^-63 + |f| 2^-107) turns.  A frequency f enters as f mod 2 pi."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import chunked_gated_delta_fwd_gb300 as m

    return m


def _arctan_inverse(n, one):
    term, total, k, sign = one // n, 0, 1, 1
    while term:
        total += sign * (term // k)
        term, k, sign = term // (n * n), k + 2, -sign
    return total


ONE = 1 << 640
PI = 4 * (4 * _arctan_inverse(5, ONE) - _arctan_inverse(239, ONE))  # Machin's formula


def phase(f, p):
    """f p modulo a whole turn, in radians."""
    turns = Fraction(float(f)) * int(p) * Fraction(ONE, 2 * PI)
    turns -= math.floor(turns)
    return float(turns - 1 if turns > Fraction(1, 2) else turns) * 2 * math.pi


def test_the_phase_is_that_of_64_bits_where_those_have_it():
    for f, p in ((1.0, 3), (-0.7, 1000), (1e-3, -77)):
        assert abs(math.remainder(phase(np.float32(f), p) - float(np.float32(f)) * p, 2 * math.pi)) < 1e-9


FREQS = [
    [1.0, -1.0, 1e9, -1e9, 1e12, 3e14, 9e15, 1.8e16],          # up to where half a turn passes 2^53
    [3e17, -3e17, 1e18, 7.7e18, -2e19, 1e20, 1e21, -1e22],      # far past it
    [-0.7, -1e-3, -1e-30, 1e-38, -1e-45, 6.2831855, -40.5, 0.5],
]


@pytest.mark.parametrize("freqs", FREQS, ids=["large", "larger", "small and negative"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
def test_frequencies_of_any_size(kda, freqs, interleaved):
    f = torch.tensor(freqs)
    pos = torch.tensor([0, 1, -1, 2, 1000, -12345, 100000, (1 << 20) + 3, -(1 << 31), (1 << 31) - 1],
                       dtype=torch.int64).to(torch.int32)
    n, F = len(pos), len(f)
    x = torch.randn(n, 2, 128, generator=torch.Generator().manual_seed(3))
    got, _ = kda.qk_norm_rope(x.cuda(), x.cuda(), pos.cuda(), f.cuda(), eps=None,
                              interleaved=interleaved)
    got, y = got.cpu().double().numpy(), x.double().numpy()
    lo, hi = (slice(0, 2 * F, 2), slice(1, 2 * F, 2)) if interleaved else (slice(0, F), slice(F, 2 * F))
    a, b = y[..., lo], y[..., hi]
    ang = np.array([[phase(z, p) for z in f] for p in pos.tolist()])[:, None, :]
    r = np.hypot(a, b)
    p64, f64 = np.abs(pos.double().numpy())[:, None, None], np.abs(f.double().numpy())
    bound = (32 * 2.0 ** -24 + 2 * math.pi * p64 * (2.0 ** -63 + f64 * 2.0 ** -107)) * r + 1e-37
    for part, ref in ((lo, a * np.cos(ang) - b * np.sin(ang)), (hi, a * np.sin(ang) + b * np.cos(ang))):
        err = np.abs(got[..., part] - ref)
        assert np.all(err <= bound), float(np.max(err / bound))
    assert np.array_equal(got[..., 2 * F:], y[..., 2 * F:])
