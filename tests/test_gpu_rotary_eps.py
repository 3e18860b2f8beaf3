"""Head norms whose mean square and eps add up to less than nothing: a root of a negative number."""
import pytest
import torch

import convolution_forward_amd as cf
import mixer_ref
import scan_ref as ref
from test_gpu_mixer import BF, DEV, F32, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("eps", [-0.5, -1e-30, -1e30])
def test_negative_eps(eps, dtype):
    """NaN for the heads whose sum is negative, by the definition, and for no others."""
    q, w = rnd((6, 2, 64), 1, dtype), rnd(64, 2, dtype)
    q[1] *= 1e-3
    q[2, 0] *= 1e-20
    q[3, 1] = 0
    pos, f = torch.arange(6), cf.rotary_frequencies(64, device="cpu")[0]
    got = cf.rotary(q.to(DEV), pos.to(DEV), f.to(DEV), q_weight=w.to(DEV), eps=eps).cpu()
    mean = q.double().square().mean(-1)
    bad = mean + torch.tensor(eps, dtype=F32).double() < 0
    assert bad.any() and torch.isnan(got[bad]).all()
    if not bad.all():
        # Heads whose mean is far above eps: the sum's rounding is in the bound.
        want, bound = ref.rotary(q, pos, f, w, eps, False, 1.0)
        fine = ~bad & (mean > 10 * abs(eps))
        mixer_ref.check(got[fine], want[fine], bound[fine], "others", dtype)
