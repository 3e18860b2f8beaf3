"""The selective scan of channels by tiles where a row's end lies inside a thread's piece: channel and state counts that are
whole 16 bytes, and not whole pieces. What lies behind a row and behind the last one is neither used nor written."""
import pytest
import torch

import convolution_forward_amd as cf
import mixer_ref
import scan_ref as ref
from mixer_ref import seqs
from test_gpu_mixer import BF, DEV, F32, rnd
from test_gpu_scan import AUTO, TILED, channel_inputs, gpu

pytestmark = pytest.mark.gpu
GUARD = 64
MARK = -77.0

# fp32 with up to 8 states takes pieces of eight channels, with 17 to 32 pieces of eight states; the last ones are whole.
SIZES = [(F32, 12, 1, 8), (F32, 4, 1, 8), (F32, 20, 1, 4), (F32, 24, 2, 8), (F32, 36, 3, 8), (F32, 68, 1, 8), (F32, 8, 2, 20),
         (F32, 8, 1, 28), (F32, 20, 1, 16), (BF, 24, 1, 8), (BF, 12, 1, 16), (BF, 8, 2, 24), (F32, 16, 1, 8), (F32, 8, 1, 32)]


def behind(t, pitch):
    """t's rows `pitch` values apart, in a buffer where NaN lies behind each row and behind the last."""
    rows = t.flatten(1)
    flat = torch.full((rows.shape[0] * pitch + GUARD,), float("nan"), dtype=t.dtype, device=DEV)
    flat[:rows.shape[0] * pitch].view(-1, pitch)[:, :rows.shape[1]] = rows.to(DEV)
    strides = (pitch,) + t.stride()[1:]
    return flat.as_strided(t.shape, strides)


@pytest.mark.parametrize("dtype,C,G,N", SIZES, ids=str)
@pytest.mark.parametrize("lens", [[40, 1, 0, 90], [700, 300]], ids=str)
@pytest.mark.parametrize("variant", [AUTO, TILED])
@pytest.mark.parametrize("room", [0, 8], ids=["rows in a run", "rows apart"])
def test_ends_inside_pieces(dtype, C, G, N, lens, variant, room):
    ins, st = channel_inputs(sum(lens), C, G, N, dtype, 30 + C + N), rnd((len(lens), C, N), 31)
    y0, by, h0, bh = ref.channels(*ins, True, lens, st)
    x, dt, a, b, c, skip, gate, bias = ins
    x, dt, gate = (behind(t, C + room) for t in (x, dt, gate))
    b, c = (behind(t, G * N + room) for t in (b, c))
    a, skip, bias, st = gpu((a, skip, bias, st))
    tokens, pitch = sum(lens), C + room
    flat = torch.full((GUARD + tokens * pitch + GUARD,), MARK, dtype=dtype, device=DEV)
    rows = flat[GUARD:GUARD + tokens * pitch].view(tokens, pitch)
    new = torch.full_like(st, float("nan"))
    y = cf.selective_scan(x, dt, a, b, c, skip=skip, gate=gate, dt_bias=bias, dt_softplus=True, seq_offsets=seqs(lens, DEV),
                          initial_state=st, final_state=new, out=rows[:, :C], variant=variant)
    mixer_ref.check(y, y0, by, "y", dtype)
    mixer_ref.check(new, h0, bh, "state", F32)
    assert (flat[:GUARD] == MARK).all() and (flat[-GUARD:] == MARK).all(), "written outside the output"
    assert (rows[:, C:] == MARK).all(), "written behind a row"
