"""Rotation at far positions: the angle is position times frequency exactly, as far as that product fits 53 bits."""
from fractions import Fraction
import math

import pytest
import torch

import convolution_forward_amd as cf
from mixer_ref import U
from test_gpu_mixer import DEV, F32

pytestmark = pytest.mark.gpu
# Of 2 pi, 50 decimals.
TURN = Fraction(628318530717958647692528676655900576839433879875021, 10 ** 50)
FREQUENCIES = [1.0, 0.5, 0.0625] + [10000.0 ** (-i / 8) for i in range(1, 8)] + [-0.3, 1.7, 0.0]


def turned(positions, frequencies):
    """cos and sin of the exact product, reduced exactly, in 64 bits."""
    out = torch.empty(len(positions), 2, len(frequencies), dtype=torch.float64)
    for i, p in enumerate(positions):
        for j, f in enumerate(frequencies.tolist()):
            angle = p * Fraction(f)
            rest = float(angle - TURN * (angle // TURN))
            out[i, 0, j], out[i, 1, j] = math.cos(rest), math.sin(rest)
    return out


def check(positions, frequencies, dtype, interleaved):
    """Heads of pairs (1, 0) come back as pairs (cos, sin).

    The reduced angle x, |x| <= 0.83, is rounded to fp32 (u / 2). cos: the rounding of z = x^2 (u z / 2 = 0.35 u), of the
    last sum (u / 2), of the one before times z (0.17 u) and of the others (0.02 u), and the series' rest (2^-28 = 0.06 u):
    1.6 u. sin: less. The products with 1 and 0 are exact.
    """
    n = len(frequencies)
    f = torch.tensor(frequencies, dtype=F32)
    q = torch.zeros(len(positions), 1, 2 * n, device=DEV)
    q[..., 0::2 if interleaved else 1] = 1.0
    if not interleaved:
        q[..., n:] = 0.0
    got = cf.rotary(q, torch.tensor(positions, dtype=dtype, device=DEV), f.to(DEV), interleaved=interleaved).cpu().double()[:, 0]
    got = got.unflatten(-1, (n, 2)).mT if interleaved else got.unflatten(-1, (2, n))
    assert (got - turned(positions, f)).abs().max() <= 2 * U


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
def test_positions_to_two_to_the_29(dtype, interleaved):
    """24 bits of frequency times 29 of position."""
    positions = [0, 1, -1, 2, 3, 100, 4095, 65537, 10 ** 6 + 3, 16777213, 2 ** 28 + 12345, 2 ** 29 - 1, 1 - 2 ** 29]
    positions += [2 ** 29 - 7919 * i for i in range(1, 200)]
    check(positions, FREQUENCIES, dtype, interleaved)


def test_further_positions():
    """Frequencies of few bits: the first one of a head is 1, whose product is exact as far as it is reduced."""
    positions = [s * (2 ** e + 97 * e) for e in range(29, 47) for s in (1, -1)]
    check(positions, [1.0, 0.5, 0.25, 1.5], torch.int64, False)


def test_positions_past_any_precision():
    """Bounded whatever the product is."""
    q = torch.ones(4, 1, 8, device=DEV)
    positions = torch.tensor([2 ** 63 - 1, -2 ** 63, 2 ** 55 + 1, 2 ** 50 + 1], device=DEV)
    got = cf.rotary(q, positions, torch.tensor([1.0, 1e10, 3e38, 0.1], device=DEV))
    assert got.abs().max() <= 1.5
