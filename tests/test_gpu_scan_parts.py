"""The selective scan of heads by chunks in fp32 where a product's lower parts count: one product for each output, of
numbers whose lower 16 bits are all ones, just below a half and random."""
import pytest
import torch

import convolution_forward_amd as cf
import mixer_ref
from mixer_ref import U
from test_gpu_mixer import DEV, F32, rnd
from test_gpu_scan import DIRECT, TILED

pytestmark = pytest.mark.gpu


def patterned(shape, seed, low):
    """Values of either sign and several exponents, with the lower 16 bits of their mantissas `low` (None: random)."""
    v = rnd(shape, seed)
    if low is None:
        return v
    return ((v.view(torch.int32) & -65536) | low).view(F32)


@pytest.mark.parametrize("variant", [DIRECT, TILED])
@pytest.mark.parametrize("low", [0xffff, 0x7fff, 0x8000, 0x7f80, None], ids=lambda v: "random" if v is None else hex(v))
def test_skipped_inputs(low, variant):
    """Steps of zero: y is skip x, off by u of it at most (one rounding; by chunks the products of parts that are left out, u,
    and the sum of the others, u more for each of the last two roundings)."""
    T, H, P, N = 130, 3, 32, 16
    x, skip = patterned((T, H, P), 1, low), patterned(H, 2, low)
    zero, bc, a = torch.zeros(T, H, device=DEV), rnd((T, 1, N), 3).to(DEV), torch.full((H,), -1.0, device=DEV)
    y = cf.selective_scan_heads(x.to(DEV), zero, a, bc, bc, skip=skip.to(DEV), variant=variant).cpu().double()
    want = skip.double()[:, None] * x.double()
    assert ((y - want).abs() <= (1 if variant == DIRECT else 3) * U * want.abs()).all()


@pytest.mark.parametrize("variant", [DIRECT, TILED])
@pytest.mark.parametrize("low", [0xffff, 0x7fff, 0x8000, 0x7f80, None], ids=lambda v: "random" if v is None else hex(v))
def test_lone_states(low, variant):
    """One state, steps of a power of two and a decay that forgets: y = c (d x b), three products and two of parts."""
    T, H, P = 130, 2, 32
    x, b, c = patterned((T, H, P), 4, low), patterned((T, 1, 1), 5, low), patterned((T, 1, 1), 6, low)
    dt, a = torch.full((T, H), 0.25, device=DEV), torch.full((H,), -4000.0, device=DEV)
    new = torch.zeros(1, H, P, 1, device=DEV)
    y = cf.selective_scan_heads(x.to(DEV), dt, a, b.to(DEV), c.to(DEV), final_state=new, variant=variant).cpu().double()
    h = 0.25 * x.double() * b.double()
    want = h * c.double()
    # Token by token: h and y are rounded. By chunks c b and its product with x: each 3 u as above.
    assert ((y - want).abs() <= (2 if variant == DIRECT else 6) * U * want.abs() * (1 + 8 * U)).all()
    assert ((new.cpu().double()[0, ..., 0] - h[-1]).abs() <= 3 * U * h[-1].abs()).all()
