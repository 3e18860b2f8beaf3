"""The token-mixer operators on the GPU at the edges of what they accept: layouts, ranges and sizes."""
import pytest
import torch

import convolution_forward_amd as cf
import mixer_ref as ref
from test_gpu_mixer import BF, DEV, F32, delta_inputs, rnd

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


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("taps", range(2, 9))
@pytest.mark.parametrize("channels,shift", [(64, 0), (68, 0), (64, 4), (68, 4), (66, 2)])
def test_conv_taps(taps, channels, shift, dtype):
    """Every number of taps, four channels a thread and one, the weights `shift` values past an aligned address."""
    lens = [40, 1, 0, 70]
    x, w = rnd((sum(lens), channels), 65, dtype), rnd((channels, taps), 66, dtype, 0.5)
    b, st = rnd(channels, 67), rnd((4, taps - 1, channels), 68, dtype)
    wd = torch.cat([torch.zeros(shift, dtype=dtype), w.flatten()]).to(DEV)[shift:].view(channels, taps)
    fin = torch.zeros_like(st, device=DEV)
    y = cf.causal_conv1d(x.to(DEV), wd, bias=b.to(DEV), activation="silu", seq_offsets=ref.seqs(lens, DEV),
                         initial_state=st.to(DEV), final_state=fin)
    y0, bound, new = ref.conv(x, w, b, True, lens, st)
    ref.check(y, y0, bound, "y")
    assert torch.equal(fin.cpu().double(), new), "state"
