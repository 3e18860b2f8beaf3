"""The token-mixer operators on the GPU at the edges of what they accept: layouts, ranges and sizes."""
import pytest
import torch

import convolution_forward_amd as cf
import mixer_ref as ref
from test_gpu_mixer import BF, DEV, E4, F32, I8, check_norm, delta_inputs, rnd

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
@pytest.mark.parametrize("qdt", [I8, E4])
@pytest.mark.parametrize("width", [300, 3000, 40000])
def test_norm_without_eps(width, qdt, dtype):
    """Rows of zeros have scale 0 and q 0; rows whose squares leave fp32's range are normed like others."""
    x = rnd((6, width), 22, dtype)
    x[0] = 0
    x[1] = -0.0
    x[2] *= 1e-22
    x[3] *= 1e-36
    x[4] = 0
    x[4, width - 1] = -1e-38
    w = rnd(width, 23, dtype)
    q, s, _ = cf.rms_norm_q8(x.to(DEV), w.to(DEV), eps=0.0, out_dtype=qdt)
    assert (s[:2] == 0).all() and (q[:2].to(F32) == 0).all()
    check_norm(q[2:], s[2:], None, x[2:], w, None, 0.0, qdt)


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


def overflow_inputs(which, dtype):
    """Finite inputs, keys not normalised, that pass 32 bits at some token: (q, k, v, g, beta, tokens up to which the
    rule is a contraction, tokens up to which a 64-bit evaluation stays inside 32 bits, tokens from which it does not)."""
    q, k, v, g, beta = delta_inputs(100, 1, 2, 64, 32, dtype, 380, unit=True)
    g, k = torch.zeros_like(g), k.float()
    if which == "products":             # of the keys of tokens 20 and 40
        k[20], k[40] = 2e19, 2e19
        beta[20], beta[40] = 1e-30, 1
        tame, fine, over = 20, 40, 41
    elif which == "growth":             # of the state, by 5e4 a token
        k[20:] *= 240
        beta[20:] = 1
        tame, fine, over = 20, 28, 32
    else:                               # of the triangle's inverse: 1e22 by token 16, then keys of 1e20
        k[4:16] *= 25
        k[16:24] *= 1e-3
        k[24:] *= 1e20
        beta[4:] = 1
        tame, fine, over = 4, 24, 26
    return q, k.to(dtype), v, g, beta, tame, fine, over


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("variant", [cf.VARIANT_DIRECT, cf.VARIANT_TILED])
@pytest.mark.parametrize("which", ["products", "growth", "inverse"])
def test_delta_overflow_reaches_no_earlier_token(which, variant, dtype):
    q, k, v, g, beta, tame, fine, over = overflow_inputs(which, dtype)
    T = q.shape[0]
    other = delta_inputs(T, 1, 2, 64, 32, dtype, 390, unit=True)
    three = [torch.cat([b, a, b]).to(DEV) for a, b in zip((q, k, v, g, beta), other)]
    fin = torch.zeros(3, 2, 64, 32, device=DEV)
    o = cf.gated_delta_rule(*three, scale=0.125, seq_offsets=ref.seqs([T] * 3, DEV), final_state=fin, variant=variant).cpu()
    good = torch.isfinite(o)
    assert good[:T + fine].all() and good[2 * T:].all() and torch.isfinite(fin[[0, 2]]).all()
    assert not good[T + over:2 * T].any() and not torch.isfinite(fin[1]).any()
    o0, bo, _, _ = ref.delta(q[:tame], k[:tame], v[:tame], g[:tame], beta[:tame], 0.125, False, [tame], None)
    ref.check(o[T:T + tame], o0, bo, "o before")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("variant", [cf.VARIANT_DIRECT, cf.VARIANT_TILED])
def test_delta_outputs_hold_32_bits(variant, dtype):
    """One key direction and beta 1: each token's value replaces the row it is written to, so o = scale v, as the sum of
    the old row (some 1000) and its negative. 33 roundings on the way, of terms no larger than those two: the rows and U
    in three parts, P likewise (4), the products of the parts (3, 3, 6, 12), Y, its factor and U in three parts."""
    T, D, Dv = 70, 64, 48
    q = torch.zeros(T, 1, D)
    q[..., 0] = 1
    v = rnd((T, 1, Dv), 371, std=0.05).to(dtype)
    g, beta = torch.zeros(T, 1), torch.ones(T, 1)
    state = torch.zeros(1, 1, D, Dv)
    state[0, 0, 0] = 600 + 400 * torch.rand(Dv, generator=torch.Generator().manual_seed(372))
    scale = torch.tensor(0.7).item()        # 24 significant bits
    o = cf.gated_delta_rule(q.to(dtype).to(DEV), q.to(dtype).to(DEV), v.to(DEV), g.to(DEV), beta.to(DEV), scale=scale,
                            initial_state=state.to(DEV), variant=variant)
    bound = 33 * ref.U * scale * (state[0, 0, 0].double() + 2 * v.double().abs())
    ref.check(o, scale * v.double(), bound, "o")


@pytest.mark.parametrize("m", [2, 20, 40])
def test_product_of_many_channels(m):
    """More channels than the few-token form's grid holds (2^27), or a grid of small tiles; sums of 8 are exact."""
    n, k = 2 ** 27 + 40, 8
    gen = torch.Generator(device=DEV).manual_seed(410)
    x, w = (torch.randint(-127, 128, (rows, k), generator=gen, device=DEV, dtype=I8) for rows in (m, n))
    y = cf.matmul_q8(x, torch.ones(m, device=DEV), w, torch.ones(n, device=DEV))
    for at in range(0, n, 2 ** 24):
        part = slice(at, at + 2 ** 24)
        assert torch.equal(y[:, part], (x.float() @ w[part].float().t()).to(BF))


def test_count_of_sequences_is_not_cut():
    """2^32 + 1 empty sequences are more than the library counts, not one."""
    with pytest.raises(ValueError, match="sequences"):
        cf.causal_conv1d(torch.empty(2 ** 32 + 1, 0, 16, device=DEV), torch.ones(16, 2, device=DEV))
