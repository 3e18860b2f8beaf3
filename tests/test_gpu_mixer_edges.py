"""The token-mixer operators on the GPU at the edges of what they accept: layouts, ranges and sizes."""
import pytest
import torch

import convolution_forward_amd as cf
from test_gpu_mixer import BF, DEV, delta_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("make", [lambda n: torch.zeros(1, dtype=torch.uint8, device=DEV).expand(n),
                                  lambda n: torch.zeros(2 * n, dtype=torch.uint8, device=DEV)[::2],
                                  lambda n: torch.zeros(n, dtype=torch.float32, device=DEV)],
                         ids=["expanded", "strided", "float32"])
def test_workspace_is_contiguous_bytes(make):
    """A view whose values are not the bytes it spans is refused: the kernels would write past or between them."""
    q, k, v, g, beta = (t.to(DEV) for t in delta_inputs(100, 1, 2, 64, 32, BF, 400))
    n = cf.delta_rule_workspace(100, 1, 1, 2, 64, 32, variant=cf.VARIANT_TILED)
    with pytest.raises(ValueError, match="workspace"):
        cf.gated_delta_rule(q, k, v, g, beta, workspace=make(n), variant=cf.VARIANT_TILED)
    o = cf.gated_delta_rule(q, k, v, g, beta, workspace=torch.empty(n, dtype=torch.uint8, device=DEV),
                            variant=cf.VARIANT_TILED)
    assert torch.equal(o, cf.gated_delta_rule(q, k, v, g, beta, variant=cf.VARIANT_TILED))
