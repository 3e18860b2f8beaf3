"""The selective scans where factors of a result lie near the ends of fp32's range and the result does not."""
import pytest
import torch

import convolution_forward_amd as cf
from test_gpu_mixer import BF, F32, rnd
from test_gpu_scan import DIRECT, TILED, check

pytestmark = pytest.mark.gpu

# (step, decay of a token as an exponent, size of x, size of c . b). exp(-1.15 x 32) is 2^-53: half a chunk's decay.
RANGES = [(0.1, 1.15, 1.0, 5e23), (0.1, 3.0, 1.0, 5e23), (0.1, 1.15, 1.0, 5e-26), (1e24, 1.15, 1e-24, 1.0), (1e24, 3.0, 1e-24, 1e20),
          (1e-30, 1.15, 1e20, 1e10), (1e-30, 3.0, 1e20, 1e10)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("step,decay,x,cb", RANGES, ids=str)
@pytest.mark.parametrize("variant", [DIRECT, TILED])
def test_factors_near_the_ends(step, decay, x, cb, variant, dtype):
    """Every c . b, state and output is far inside fp32's range; the step, or c . b times half a chunk's decay, is not."""
    if variant == TILED and step * cb > 3e38:
        heads = []      # by chunks d c . b is a number of its own, here 1e24 x 1e20: past fp32's largest, 3.4e38
    else:
        heads = [(cf.selective_scan_heads, 64, (16,), (2,))]
    lens = [150, 64]
    T = sum(lens)

    def near(shape, seed, size):        # around size, of one sign
        return ((1.0 + 0.2 * rnd(shape, seed).clamp(-3, 3)) * size).to(dtype)
    dt, skip = near((T, 2), 1, step), rnd(2, 2)
    for fn, N, width, rates in heads + [(cf.selective_scan, 32, (), (2, 32))]:
        b, c = (near((T, 1, N), seed, (cb / N) ** 0.5) for seed in (3, 4))
        ins = [near((T, 2) + width, 5, x), dt, torch.full(rates, -decay / step), b, c, skip, None, None]
        check(fn, ins, lens, None, variant, softplus=False)
