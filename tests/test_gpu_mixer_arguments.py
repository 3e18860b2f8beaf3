"""Arguments of the token-mixer calls as Python passes them: variants past 32 bits, and positions of batches."""
import pytest
import torch

import convolution_forward_amd as cf
from test_gpu_mixer import BF, DEV, rnd
from test_gpu_scan import channel_inputs, gpu, head_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("variant", [2 ** 32, 2 ** 32 + 1, -2 ** 32, 2 ** 33 + 2, -1, 2 ** 31 - 1])
def test_variants_that_there_are_not(variant):
    """None is cut to 32 bits and taken for one that there is."""
    x, dt, a, b, c, *_ = gpu(channel_inputs(20, 24, 2, 16, BF, 1))
    with pytest.raises(ValueError):
        cf.selective_scan(x, dt, a, b, c, variant=variant)
    x, dt, a, b, c, *_ = gpu(head_inputs(20, 4, 32, 2, 64, BF, 1))
    with pytest.raises(ValueError):
        cf.selective_scan_heads(x, dt, a, b, c, variant=variant)
    q, g = rnd((20, 2, 32), 2, BF).to(DEV), torch.zeros(20, 2, device=DEV)
    with pytest.raises(ValueError):
        cf.gated_delta_rule(q, q, q, g, g, variant=variant)
    w, s = torch.zeros(16, 64, dtype=torch.int8, device=DEV), torch.ones(16, device=DEV)
    with pytest.raises(ValueError):
        cf.matmul_q8(w, s, w, s, variant=variant)


def test_positions_of_a_batch():
    """[batch, length] as well as one axis; what is not contiguous is refused."""
    q = rnd((3, 5, 2, 32), 3, BF).to(DEV)
    positions, f = torch.randint(0, 1000, (3, 5), device=DEV), cf.rotary_frequencies(32)[0]
    y = cf.rotary(q, positions, f)
    assert torch.equal(y, cf.rotary(q, positions.flatten(), f))
    assert torch.equal(y.flatten(0, 1), cf.rotary(q.flatten(0, 1), positions.flatten().int(), f))
    same = torch.arange(5, device=DEV).expand(3, 5)
    with pytest.raises(ValueError):
        cf.rotary(q, same, f)
    assert torch.equal(cf.rotary(q, same.contiguous(), f)[1], cf.rotary(q[1], same[1], f))
