"""Rates at fp32's end: a state forgotten at each token with a step, and kept at a token without one."""
import pytest
import torch

import convolution_forward_amd as cf
from test_gpu_mixer import BF, F32, rnd
from test_gpu_scan import DIRECT, TILED, channel_inputs, check, head_inputs, run

pytestmark = pytest.mark.gpu
STRONG = -5000.0        # times a step of 0.1 or more: exp is 0 in 64 bits' first 200 places too


@pytest.mark.parametrize("rate", [-float("inf"), torch.finfo(F32).min, -3e38])
@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("variant", [DIRECT, TILED])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fn,ins,shape", [(cf.selective_scan, channel_inputs(210, 24, 2, 16, BF, 61), (24, 16)),
                                          (cf.selective_scan, channel_inputs(210, 9, 1, 5, BF, 62), (9, 5)),
                                          (cf.selective_scan_heads, head_inputs(210, 4, 32, 2, 64, BF, 63), (4, 32, 64)),
                                          (cf.selective_scan_heads, head_inputs(210, 2, 5, 1, 3, BF, 64), (2, 5, 3))],
                         ids=["channels", "few channels", "heads", "few heads"])
def test_rates_at_the_end(fn, ins, shape, dtype, variant, softplus, rate):
    """The same bits as a rate that is strong enough, which is what the definition gives; some tokens' steps are zero."""
    x, dt, a, b, c, skip, gate, bias = ins
    x, b, c, gate = (t.to(dtype) for t in (x, b, c, gate))
    dt = (0.2 + dt.float().abs()).to(dtype)
    dt[3:9] = dt[100:131] = dt[205:] = -float("inf") if softplus else 0.0
    hit = torch.rand(a.shape, generator=torch.Generator().manual_seed(5)) < 0.5
    hit.view(-1)[0] = True
    lens, st = [130, 80], rnd((2,) + shape, 65)
    got = []
    # (The definition's bounds take finite sums: softplus of -200, 1e-87, is the step of zero there. Here it has the same bits.)
    for r, zero in ((STRONG, -200.0), (STRONG, -float("inf")), (rate, -float("inf"))):
        steps = torch.where(torch.isinf(dt), torch.tensor(zero, dtype=dtype), dt)
        inputs = [x, steps, torch.where(hit, torch.tensor(r), a), b, c, skip, gate, None]
        got.append(run(fn, inputs, lens, st, variant, softplus))
        if zero == -200.0:
            check(fn, inputs, lens, st, variant, softplus)
    for y, new in got[1:]:
        assert torch.equal(y, got[0][0]) and torch.equal(new, got[0][1])
