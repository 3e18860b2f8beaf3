"""Stretched frequencies where all of them are slow: none makes a turn in the positions trained on."""
import math

import pytest
import torch

import convolution_forward_amd as cf


@pytest.mark.parametrize("scaling", ["parts", "wavelength"])
@pytest.mark.parametrize("trained,slow", [(6, 1.0), (1, 1.0), (100, 16.0), (7, 7 / (2 * math.pi))])
def test_all_slow_frequencies_are_divided(scaling, trained, slow):
    """The fastest, 1 radian a position, makes trained / 2 pi turns: at most `slow` here, so it is divided as the others are."""
    f, _ = cf.rotary_frequencies(16, device="cpu")
    g, _ = cf.rotary_frequencies(16, scaling=scaling, factor=4.0, trained=trained, fast=32.0, slow=slow, device="cpu")
    assert trained / (2 * math.pi) <= slow and torch.equal(g, f / 4)


@pytest.mark.parametrize("trained", [8, 20, 201])
def test_the_fastest_between_the_bounds_is_not_divided_whole(trained):
    """A turn or more of the fastest frequency: it is on the ramp or before it, and the order of frequencies stays."""
    g, _ = cf.rotary_frequencies(16, scaling="parts", factor=4.0, trained=trained, fast=32.0, slow=1.0, device="cpu")
    assert g[0] > 0.25 and (g[1:] < g[:-1]).all() and math.isclose(g[-1], 10000.0 ** (-7 / 8) / 4, rel_tol=1e-6)
