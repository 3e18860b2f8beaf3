"""The token-mixer operators on the GPU against their definitions in 64 bits (mixer_ref.py), at the sizes, layouts and
values where they can go wrong."""
import pytest
import torch

import convolution_forward_amd as cf
import mixer_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, I8, E4 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn


def rnd(shape, seed, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def padded(t, extra, fill=float("nan")):
    """The same values on the GPU as a view of rows `extra` longer, the rest holding `fill`."""
    big = torch.full(t.shape[:-1] + (t.shape[-1] + extra,), fill, dtype=torch.float32).to(t.dtype)
    big[..., :t.shape[-1]] = t
    return big.to(DEV)[..., :t.shape[-1]]


# ---- norm ------------------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("qdt", [I8, E4])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (2, 64), (5, 513), (4, 1000), (7, 2048), (2, 2880), (3, 4097),
                                        (2, 8192), (1, 16384), (2, 16400), (1, 40000)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(rows, width, dtype, qdt, residual):
    x, w = rnd((rows, width), 1, dtype), rnd(width, 2, dtype) * 0.2 + 1
    r = rnd((rows, width), 3, dtype, 3.0) if residual else None
    w = w.to(dtype)
    q, s, h = cf.rms_norm_q8(x.to(DEV), w.to(DEV), residual=None if r is None else r.to(DEV), eps=1e-5, out_dtype=qdt)
    check_norm(q, s, h, x, w, r, 1e-5, qdt)


def check_norm(q, s, h, x, w, r, eps, qdt):
    wh, y, rel = ref.norm(x, w, r, eps)
    if r is not None:
        assert torch.equal(h.cpu(), wh)
    top = y.abs().amax(-1)
    ref.check(s, top / ref.QMAX[qdt], top / ref.QMAX[qdt] * (rel + 2 * ref.U), "scale", F32)
    want = torch.where(top[:, None] > 0, y / top[:, None] * ref.QMAX[qdt], 0.0)
    ref.check(q, want, want.abs() * (2 * rel + 4 * ref.U), "q", qdt)


def test_norm_many_rows():
    """More rows than one launch takes: the same as a call on the rows round its end."""
    rows = 2 ** 21 + 3
    x = torch.arange(rows * 8, device=DEV).remainder(8191).sub(4000).to(BF).reshape(rows, 8)
    w = rnd(8, 14, BF).to(DEV)
    q, s, h = cf.rms_norm_q8(x, w, residual=x.flip(0))
    some = slice(2 ** 21 - 4, None)
    for a, b in zip((q, s, h), cf.rms_norm_q8(x[some], w, residual=x.flip(0)[some])):
        assert torch.equal(a[some], b)


def test_norm_strided_and_in_place():
    """Rows with a pitch (NaN between them), 2-byte alignment only, and the sum written over the residual."""
    for width, extra in ((256, 8), (256, 1), (1030, 3)):
        x, r, w = rnd((6, width), 11, BF), rnd((6, width), 12, BF), rnd(width, 13, BF)
        xs, rs = padded(x, extra), padded(r, extra)
        out = torch.full((6, width + 5), 77, dtype=I8, device=DEV)
        q, s, h = cf.rms_norm_q8(xs, w.to(DEV), residual=rs, sum_out=rs, out=out[:, :width])
        check_norm(q.contiguous(), s, h.contiguous(), x, w, r, 1e-6, I8)
        assert (out[:, width:] == 77).all()
        assert torch.isnan(rs._base[:, width:]).all()
    shifted = torch.cat([rnd(1, 1, BF), rnd(4 * 128, 14, BF)]).to(DEV)[1:].view(4, 128)       # 2 bytes past alignment
    q, s, _ = cf.rms_norm_q8(shifted, w.to(DEV)[:128], out_dtype=E4)
    check_norm(q, s, None, shifted.cpu(), w[:128], None, 1e-6, E4)
    x3 = rnd((2, 3, 128), 15, BF)
    q, s, _ = cf.rms_norm_q8(x3.to(DEV), w.to(DEV)[:128])
    assert q.shape == (2, 3, 128) and s.shape == (2, 3)
    check_norm(q.view(6, 128), s.view(6), None, x3.view(6, 128), w[:128], None, 1e-6, I8)


@pytest.mark.parametrize("qdt", [I8, E4])
def test_norm_special_rows(qdt):
    x = rnd((7, 300), 21, BF)
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 299] = float("nan")
    x[3] = 1e-30
    x[4] = 3e38                    # the square overflows
    x[5, :] = 0
    x[5, 17] = 2.0                 # a single value
    w = torch.ones(300, dtype=BF)
    q, s, _ = cf.rms_norm_q8(x.to(DEV), w.to(DEV), out_dtype=qdt)
    q, s = q.cpu().to(F32), s.cpu()
    assert s[0] == 0 and (q[0] == 0).all()
    for bad in (1, 2, 4):
        assert torch.isnan(s[bad]) and (q[bad] == 0).all()
    assert torch.isfinite(s[3]) and s[3] > 0 and (q[3] == ref.QMAX[qdt]).all()
    assert q[5, 17] == ref.QMAX[qdt] and (q[5].count_nonzero() == 1)
    check_norm(q[5:].to(qdt), s[5:], None, x[5:], w, None, 1e-6, qdt)
    w[3] = float("nan")
    _, s, _ = cf.rms_norm_q8(x.to(DEV), w.to(DEV), out_dtype=qdt)
    assert torch.isnan(s).all()


def test_norm_no_rows():
    q, s, h = cf.rms_norm_q8(torch.empty(0, 64, device=DEV), torch.ones(64, device=DEV))
    assert q.shape == (0, 64) and s.shape == (0,) and h is None


# ---- product ---------------------------------------------------------------------------------------------------------


def eight(shape, seed, qdt):
    t = rnd(shape, seed, std=40.0 if qdt == I8 else 100.0)
    return t.clamp(-127, 127).round().to(I8) if qdt == I8 else t.clamp(-448, 448).to(E4)


SIZES = [(1, 1, 1), (1, 16, 64), (3, 5, 31), (2, 1000, 128), (8, 256, 4096), (16, 130, 144), (17, 64, 256), (33, 200, 100),
         (64, 96, 1040), (65, 257, 513), (128, 128, 128), (129, 300, 640), (200, 512, 2064), (256, 256, 1024),
         (300, 257, 192), (513, 520, 400), (1000, 384, 272)]


@pytest.mark.parametrize("variant", [cf.VARIANT_AUTO, cf.VARIANT_DIRECT])
@pytest.mark.parametrize("qdt", [I8, E4])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(m, n, k, qdt, variant):
    x, w = eight((m, k), m + k, qdt), eight((n, k), n + k, qdt)
    xs, ws = rnd(m, 31).abs() * 0.05, rnd(n, 32).abs() * 0.01
    for bias, dt in ((None, F32), (rnd(n, 33), BF)):
        y = cf.matmul_q8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV), bias=None if bias is None else bias.to(DEV),
                         out_dtype=dt, variant=variant)
        want, bound = ref.product(x, xs, w, ws, bias)
        ref.check(y, want, bound, f"product {m}x{n}x{k} {qdt} {dt}")


@pytest.mark.parametrize("qdt", [I8, E4])
@pytest.mark.parametrize("k", [288, 413])
@pytest.mark.parametrize("m,n", [(40, 100), (60, 8402), (130, 8300), (250, 12901), (500, 16000), (1000, 16008)])
def test_product_tiles(m, n, k, qdt):
    """A size for each tile, the largest one's last, with rows, channels and K that it does not divide."""
    x, w = eight((m, k), 51, qdt), eight((n, k), 52, qdt)
    xs, ws, bias = rnd(m, 53).abs() * 0.05, rnd(n, 54).abs() * 0.01, rnd(n, 55)
    for dt in (F32, BF):
        y = cf.matmul_q8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV), bias=bias.to(DEV), out_dtype=dt)
        want, bound = ref.product(x, xs, w, ws, bias)
        ref.check(y, want, bound, f"product {m}x{n}x{k} {qdt} {dt}")


@pytest.mark.parametrize("qdt", [I8, E4])
@pytest.mark.parametrize("m", [5, 70, 300])
def test_product_strided(qdt, m):
    """Operand rows with a pitch of every alignment, K inside a 16-byte piece, what lies between rows never used."""
    n, k = 150, 200
    x, w = eight((m, k), 41, qdt), eight((n, k), 42, qdt)
    xs, ws = rnd(m, 43).abs(), rnd(n, 44).abs() * 0.01
    want, bound = ref.product(x, xs, w, ws, None)
    fill = 127.0 if qdt == I8 else float("nan")
    for ex, ew in ((8, 8), (8, 56), (1, 0), (0, 3), (4, 4), (56, 56)):
        px, pw = padded(x, ex, fill), padded(w, ew, fill)
        out = torch.full((m, n + 7), 5.0, device=DEV)
        y = cf.matmul_q8(px, xs.to(DEV), pw, ws.to(DEV), out=out[:, :n])
        ref.check(y, want, bound, f"pitches {k + ex}, {k + ew}")
        assert (out[:, n:] == 5.0).all()


def test_product_largest_sums_are_exact():
    """Every product +-127^2 with K at the limit: 32-bit sums, no wrap."""
    for k in (4096, 131071):
        x = torch.full((3, k), 127, dtype=I8)
        w = torch.full((5, k), 127, dtype=I8)
        w[1], w[2, ::2] = -127, -127
        y = cf.matmul_q8(x.to(DEV), torch.ones(3, device=DEV), w.to(DEV), torch.ones(5, device=DEV), out_dtype=F32)
        want = (x.double() @ w.double().t()).float()
        assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("m", [4, 100])
def test_product_special_values(m):
    """A NaN or infinite operand or scale stays in its row or column."""
    x, w = eight((m, 256), 51, E4), eight((40, 256), 52, E4)
    x = x.float()
    x[2, 7] = float("nan")
    x = x.to(E4)
    xs, ws = torch.ones(m), torch.ones(40)
    xs[1], ws[3] = float("inf"), float("nan")
    y = cf.matmul_q8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV), out_dtype=F32).cpu()
    assert torch.isnan(y[2]).all() and torch.isnan(y[:, 3]).all() and torch.isinf(y[1, [0, 4, 39]]).all()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[1], keep[2], keep[:, 3] = False, False, False
    assert torch.isfinite(y[keep]).all()


def test_product_no_rows():
    y = cf.matmul_q8(torch.empty(0, 64, dtype=I8, device=DEV), torch.empty(0, device=DEV),
                     torch.ones(8, 64, dtype=I8, device=DEV), torch.ones(8, device=DEV))
    assert y.shape == (0, 8)


# ---- causal convolution ----------------------------------------------------------------------------------------------

LENS = [[1], [5], [0, 1, 40, 0, 2, 17], [1] * 70, [16, 32, 15, 17], [300], [0, 0, 0]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("channels,taps", [(1, 2), (24, 4), (8, 8), (2048, 4), (2056, 3), (37, 4), (130, 5)])
def test_conv(lens, channels, taps, dtype):
    T, n = sum(lens), len(lens)
    x, w, b = rnd((T, channels), 61, dtype), rnd((channels, taps), 62, dtype, 0.5), rnd(channels, 63)
    st = rnd((n, taps - 1, channels), 64, dtype)
    for bias, act, state in ((b, "silu", st), (None, None, None)):
        y0, bound, new = ref.conv(x, w, bias, act == "silu", lens, state)
        fin = torch.full((n, taps - 1, channels), 9.0, dtype=dtype, device=DEV)
        y = cf.causal_conv1d(x.to(DEV), w.to(DEV), bias=None if bias is None else bias.to(DEV), activation=act,
                             seq_offsets=ref.seqs(lens, DEV), initial_state=None if state is None else state.to(DEV),
                             final_state=fin)
        ref.check(y, y0, bound, "y")
        assert torch.equal(fin.cpu().double(), new), "state"


def test_conv_slots_in_place():
    """States in place through slots: sequences shorter than the window keep old rows, a slot of -1 or past the end
    starts from zeros and keeps nothing, unnamed slots stay as they are."""
    lens, C, taps = [2, 0, 1, 5, 33, 4], 264, 4
    slots = [4, 0, 7, -1, 2, 8]
    x, w = rnd((sum(lens), C), 71, BF), rnd((C, taps), 72, BF)
    pool = rnd((8, taps - 1, C), 73, BF)
    start = torch.stack([pool[s] if 0 <= s < 8 else torch.zeros_like(pool[0]) for s in slots])
    y0, bound, new = ref.conv(x, w, None, True, lens, start)
    dev = pool.to(DEV)
    y = cf.causal_conv1d(x.to(DEV), w.to(DEV), activation="silu", seq_offsets=ref.seqs(lens, DEV), initial_state=dev,
                         final_state=dev, slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    ref.check(y, y0, bound, "y")
    want = pool.double()
    for i, s in enumerate(slots):
        if 0 <= s < 8:
            want[s] = new[i]
    assert torch.equal(dev.cpu().double(), want)


def test_conv_strided_batch_and_steps():
    """A batch as a slice of wider rows; a sequence in one call equals the same tokens in several."""
    x, w = rnd((3, 50, 72), 81, BF), rnd((72, 4), 82, BF)
    wide = padded(x, 8)
    y = cf.causal_conv1d(wide, w.to(DEV), activation="silu")
    y0, bound, _ = ref.conv(x.view(150, 72), w, None, True, [50] * 3, None)
    ref.check(y.reshape(150, 72), y0, bound, "batch")
    state = torch.zeros(3, 3, 72, dtype=BF, device=DEV)
    parts = [cf.causal_conv1d(part.contiguous(), w.to(DEV), activation="silu", initial_state=state, final_state=state)
             for part in x.to(DEV).split([1, 2, 1, 20, 26], dim=1)]
    assert torch.equal(torch.cat(parts, 1), y)


def test_conv_special_values():
    x, w = rnd((40, 16), 91, F32), rnd((16, 4), 92, F32)
    x[10, 3], x[20, 5] = float("nan"), float("inf")
    y = cf.causal_conv1d(x.to(DEV), w.to(DEV)).cpu()
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[10:14, 3] = True
    want[20:24, 5] = True
    assert torch.equal(bad, want)
    big = torch.tensor([[-200.0, 200.0, -1e30, 1e30]], device=DEV).repeat(1, 4)
    one = torch.zeros(16, 2, device=DEV)
    one[:, 1] = 1
    y = cf.causal_conv1d(big, one, activation="silu").cpu()
    assert torch.equal(y[0, :4], torch.tensor([-0.0, 200.0, -0.0, 1e30])) and torch.isfinite(y).all()


# ---- gated delta rule ------------------------------------------------------------------------------------------------


def delta_inputs(T, Hk, Hv, Dk, Dv, dtype, seed, unit=False):
    q, k = (torch.nn.functional.silu(rnd((T, Hk, Dk), seed + i)) for i in range(2))
    if unit:
        q, k = q / q.norm(dim=-1, keepdim=True).clamp_min(1e-3), k / k.norm(dim=-1, keepdim=True).clamp_min(1e-3)
    v = rnd((T, Hv, Dv), seed + 2)
    g = -torch.nn.functional.softplus(rnd((T, Hv), seed + 3, std=2.0) - 2.0)
    beta = torch.sigmoid(rnd((T, Hv), seed + 4))
    return q.to(dtype), k.to(dtype), v.to(dtype), g, beta


def run_delta(q, k, v, g, beta, lens, states, normalize, scale=None, want_state=True, **kw):
    n, Hv, Dk, Dv = len(lens), v.shape[1], q.shape[2], v.shape[2]
    fin = torch.full((n, Hv, Dk, Dv), 7.0, device=DEV) if want_state else None
    o = cf.gated_delta_rule(q.to(DEV), k.to(DEV), v.to(DEV), g.to(DEV), beta.to(DEV), scale=scale, normalize=normalize,
                            seq_offsets=ref.seqs(lens, DEV), initial_state=None if states is None else states.to(DEV),
                            final_state=fin, **kw)
    o0, bo, s0, bs = ref.delta(q, k, v, g, beta, q.shape[2] ** -0.5 if scale is None else scale, normalize, lens, states)
    ref.check(o, o0, bo, "o")
    if want_state:
        ref.check(fin, s0, bs, "state")
    return o


VARIANTS = [cf.VARIANT_AUTO, cf.VARIANT_DIRECT]     # AUTO: by chunks wherever that form takes the sizes and pays
DELTA_LENS = [[1], [2], [63], [64], [65], [0, 1, 130, 0, 64, 3], [1] * 9, [200]]


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", DELTA_LENS, ids=str)
def test_delta_lengths(lens, dtype, variant):
    q, k, v, g, beta = delta_inputs(sum(lens), 2, 4, 64, 48, dtype, 100)
    states = rnd((len(lens), 4, 64, 48), 105, std=0.3)
    run_delta(q, k, v, g, beta, lens, states, True, variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hk,Hv,Dk,Dv", [(1, 1, 1, 1), (1, 1, 8, 16), (2, 2, 128, 128), (1, 4, 96, 80), (3, 3, 40, 33),
                                         (1, 2, 100, 130), (2, 6, 16, 256), (1, 1, 13, 7)])
def test_delta_heads(Hk, Hv, Dk, Dv, dtype, variant):
    lens = [70, 1, 90]
    q, k, v, g, beta = delta_inputs(sum(lens), Hk, Hv, Dk, Dv, dtype, 200)
    run_delta(q, k, v, g, beta, lens, None, True, variant=variant)
    q, k, v, g, beta = delta_inputs(sum(lens), Hk, Hv, Dk, Dv, dtype, 210, unit=True)
    run_delta(q, k, v, g, beta, lens, rnd((3, Hv, Dk, Dv), 215, std=0.3), False, scale=0.7, variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_padded_rows(dtype, variant):
    """Heads of 100 and 60 values in aligned rows of 104 and 64, NaN between them."""
    lens = [70, 2]
    q, k, v, g, beta = delta_inputs(72, 2, 2, 100, 60, dtype, 225)
    fin = torch.zeros(2, 2, 100, 60, device=DEV)
    o = cf.gated_delta_rule(padded(q, 4), padded(k, 4), padded(v, 4), g.to(DEV), beta.to(DEV), normalize=True,
                            seq_offsets=ref.seqs(lens, DEV), final_state=fin, variant=variant)
    o0, bo, s0, bs = ref.delta(q, k, v, g, beta, 0.1, True, lens, None)
    ref.check(o, o0, bo, "o")
    ref.check(fin, s0, bs, "state")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_many_chunks(dtype):
    """More chunks than the chip holds at once (another split of the preparation), six value heads a key head."""
    lens = [3] * 130 + [70, 0, 129] + [1] * 90
    q, k, v, g, beta = delta_inputs(sum(lens), 1, 6, 64, 16, dtype, 220)
    run_delta(q, k, v, g, beta, lens, None, True, variant=cf.VARIANT_TILED)


def test_delta_wide_heads():
    """Dk past the chunked form's limit."""
    lens = [20, 3]
    q, k, v, g, beta = delta_inputs(23, 1, 2, 200, 64, BF, 230)
    run_delta(q, k, v, g, beta, lens, None, True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("variant", VARIANTS)
def test_delta_correlated_keys(variant, dtype):
    """Nearly equal keys and beta 1: the triangular system at its worst."""
    lens = [150]
    q, k, v, g, beta = delta_inputs(150, 1, 2, 64, 32, dtype, 240)
    k = (k[:1] + 0.05 * rnd(k.shape, 241)).to(dtype)
    run_delta(q, k, v, torch.zeros_like(g), torch.ones_like(beta), lens, None, True, variant=variant)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("variant", VARIANTS)
def test_delta_gates(variant, dtype):
    """Gates of every strength: none, total (-inf, which forgets all before it, even what is not finite in no place),
    and long runs of strong ones whose sum passes what an fp32 difference resolves."""
    T = 200
    q, k, v, g, beta = delta_inputs(T, 1, 3, 64, 32, dtype, 250)
    g[:, 0] = 0.0
    g[::7, 1] = float("-inf")
    g[100, 1] = -3e38
    g[:130, 2] = -80.0
    g[130:, 2] = -0.01
    beta[::5] = 0.0
    run_delta(q, k, v, g, beta, [T], rnd((1, 3, 64, 32), 255), True, variant=variant)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("variant", VARIANTS)
def test_delta_zero_rows(variant, dtype):
    """Keys and queries of zeros (normalised: still zeros)."""
    q, k, v, g, beta = delta_inputs(100, 1, 1, 32, 32, dtype, 260)
    k[10:80], q[70:] = 0, 0
    run_delta(q, k, v, g, beta, [100], None, True, variant=variant)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("T", [1, 100])
def test_delta_nan_stays_in_its_sequence_and_head(variant, T):
    lens = [T, T, T]
    q, k, v, g, beta = delta_inputs(3 * T, 1, 2, 64, 32, BF, 270)
    v[T + T // 2, 1, 5] = float("nan")
    fin = torch.zeros(3, 2, 64, 32, device=DEV)
    o = cf.gated_delta_rule(q.to(DEV), k.to(DEV), v.to(DEV), g.to(DEV), beta.to(DEV), normalize=True,
                            seq_offsets=ref.seqs(lens, DEV), final_state=fin, variant=variant).cpu()
    bad = torch.isnan(o)
    assert bad[T + T // 2:2 * T, 1, 5].all()
    assert not bad[:T].any() and not bad[2 * T:].any() and not bad[:, 0].any() and not bad[:T + T // 2].any()
    assert not torch.isnan(fin[[0, 2]]).any() and not torch.isnan(fin[1, 0]).any()
    cols = torch.arange(32) != 5
    assert not bad[:, 1, cols].any() and not torch.isnan(fin[1, 1][:, cols]).any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("lens", [[1, 1, 1, 1, 1], [70, 0, 1, 128, 9]], ids=str)
def test_delta_slots_in_place(lens, variant, dtype):
    slots = [6, 0, -1, 3, 9]
    q, k, v, g, beta = delta_inputs(sum(lens), 2, 2, 64, 64, dtype, 280)
    pool = rnd((7, 2, 64, 64), 285, std=0.3)
    start = torch.stack([pool[s] if 0 <= s < 7 else torch.zeros_like(pool[0]) for s in slots])
    dev = pool.to(DEV)
    o = cf.gated_delta_rule(q.to(DEV), k.to(DEV), v.to(DEV), g.to(DEV), beta.to(DEV), normalize=True,
                            seq_offsets=ref.seqs(lens, DEV), initial_state=dev, final_state=dev,
                            slots=torch.tensor(slots, dtype=torch.int32, device=DEV), variant=variant)
    o0, bo, s0, bs = ref.delta(q, k, v, g, beta, 0.125, True, lens, start)
    ref.check(o, o0, bo, "o")
    want, bound = pool.double(), torch.zeros_like(pool, dtype=torch.float64)
    for i, s in enumerate(slots):
        if 0 <= s < 7:
            want[s], bound[s] = s0[i], bs[i]
    ref.check(dev, want, bound, "pool")


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("extra", [8, 3])
def test_delta_strided(variant, extra):
    """Heads as slices of wider rows, NaN between them, at 16-byte and at odd steps; outputs into a wider buffer; heads
    outermost."""
    T, Hk, Hv, D = 90, 2, 2, 64
    q, k, v, g, beta = delta_inputs(T, Hk, Hv, D, D, BF, 290)
    o0, bo, s0, bs = ref.delta(q, k, v, g, beta, 0.125, True, [T], None)
    both = torch.full((T, 3, Hk, D + extra), float("nan"), dtype=BF)
    for i, t in enumerate((q, k, v)):
        both[:, i, :, :D] = t
    both = both.to(DEV)
    out = torch.full((Hv, T, D + extra), 3.0, dtype=BF, device=DEV)
    view = out[:, :, :D].transpose(0, 1)
    cf.gated_delta_rule(both[:, 0, :, :D], both[:, 1, :, :D], both[:, 2, :, :D], g.to(DEV), beta.to(DEV), normalize=True,
                        out=view, variant=variant)
    ref.check(view, o0, bo, "o")
    assert (out[:, :, D:] == 3.0).all()


@pytest.mark.parametrize("variant", VARIANTS)
def test_delta_batch_and_steps(variant):
    """[batch, length] tensors; and a prompt in pieces down to single tokens gives what one call gives, within the
    rounding of both."""
    B, L = 2, 140
    q, k, v, g, beta = delta_inputs(B * L, 1, 2, 64, 32, F32, 300)
    q, k, v = q.to(BF).float(), k.to(BF).float(), v.to(BF).float()
    dt = BF if variant == cf.VARIANT_AUTO else F32
    four = [t.to(dt).view(B, L, *t.shape[1:]).to(DEV) for t in (q, k, v)] + [t.view(B, L, 2).to(DEV) for t in (g, beta)]
    fin = torch.zeros(B, 2, 64, 32, device=DEV)
    o = cf.gated_delta_rule(*four, normalize=True, final_state=fin, variant=variant)
    o0, bo, s0, bs = ref.delta(q, k, v, g, beta, 0.125, True, [L] * B, None)
    ref.check(o.reshape(B * L, 2, 32), o0, bo, "o")
    ref.check(fin, s0, bs, "state")
    state = torch.zeros_like(fin)
    parts = []
    for a, b in ((0, 1), (1, 2), (2, 67), (67, 68), (68, 140)):
        parts.append(cf.gated_delta_rule(*[t[:, a:b].contiguous() for t in four], normalize=True, initial_state=state,
                                         final_state=state, variant=variant))
    ref.check(torch.cat(parts, 1).reshape(B * L, 2, 32), o0, bo, "o in pieces")
    ref.check(state, s0, bs, "state in pieces")


def test_delta_no_tokens():
    """Only empty sequences: the states go over as they are."""
    st = rnd((3, 2, 32, 16), 310).to(DEV)
    fin = torch.zeros_like(st)
    z = lambda *s: torch.empty(*s, dtype=BF, device=DEV)  # noqa: E731
    zf = torch.empty(0, 2, device=DEV)
    o = cf.gated_delta_rule(z(0, 2, 32), z(0, 2, 32), z(0, 2, 16), zf, zf, seq_offsets=ref.seqs([0, 0, 0], DEV),
                            initial_state=st, final_state=fin)
    assert o.shape == (0, 2, 16) and torch.equal(st, fin)


@pytest.mark.parametrize("lens", [[1], [3, 0, 1, 2], [17] * 3, [64], [129]], ids=str)
@pytest.mark.parametrize("Hk,Hv,Dk,Dv", [(1, 1, 8, 16), (1, 2, 64, 64), (2, 4, 128, 128), (1, 3, 100, 34)])
def test_delta_by_chunks(lens, Hk, Hv, Dk, Dv):
    """The chunked form forced, single tokens and empty sequences included."""
    q, k, v, g, beta = delta_inputs(sum(lens), Hk, Hv, Dk, Dv, BF, 350)
    run_delta(q, k, v, g, beta, lens, rnd((len(lens), Hv, Dk, Dv), 355, std=0.3), True, variant=cf.VARIANT_TILED)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("which,value", [("k", float("nan")), ("k", float("inf")), ("g", float("nan")),
                                         ("g", float("inf")), ("beta", float("nan")), ("q", float("nan")),
                                         ("v", float("-inf")), ("state", float("nan"))])
def test_delta_not_finite(which, value, variant, dtype):
    """What is not finite reaches its own token and later ones of its head (q: its token only; v and the state: its
    column), never earlier tokens, other heads or other sequences."""
    lens, t = [90, 100, 40], 70
    q, k, v, g, beta = delta_inputs(sum(lens), 2, 2, 64, 32, dtype, 360)
    states = rnd((3, 2, 64, 32), 365, std=0.3)
    at = 90 + t
    if which == "state":
        states[1, 1, 7, 5] = value
    elif which in "gbeta":
        (g if which == "g" else beta)[at, 1] = value
    else:
        dict(q=q, k=k, v=v)[which][at, 1, 5] = value
    fin = torch.zeros(3, 2, 64, 32, device=DEV)
    o = cf.gated_delta_rule(q.to(DEV), k.to(DEV), v.to(DEV), g.to(DEV), beta.to(DEV), normalize=True,
                            seq_offsets=ref.seqs(lens, DEV), initial_state=states.to(DEV), final_state=fin,
                            variant=variant).cpu()
    bad = ~torch.isfinite(o)
    want = torch.zeros_like(bad)
    if which == "q":
        want[at, 1] = True
    elif which == "state":
        want[90:190, 1, 5] = True
    elif which == "v":
        want[at:190, 1, 5] = True
    else:
        want[at:190, 1] = True
    if value == float("inf") and which == "k":      # normalised: the infinite entry makes the others 0, itself NaN
        assert bad[want].any() and not bad[~want].any()
    else:
        assert torch.equal(bad, want)
    fin = fin.cpu()
    assert torch.isfinite(fin[[0, 2]]).all() and torch.isfinite(fin[1, 0]).all()
    if which == "q":
        assert torch.isfinite(fin).all()
    elif which in ("v", "state"):
        cols = torch.arange(32) != 5
        assert torch.isfinite(fin[1, 1][:, cols]).all() and not torch.isfinite(fin[1, 1][:, 5]).any()


# ---- all of them -----------------------------------------------------------------------------------------------------


def test_offsets_out_of_range_stay_in_bounds():
    """Offsets past the tokens are clamped; the sequences that are right keep their results."""
    x, w = rnd((20, 64), 320, BF).to(DEV), rnd((64, 4), 321, BF).to(DEV)
    good = cf.causal_conv1d(x, w, seq_offsets=torch.tensor([0, 12, 20], dtype=torch.int32, device=DEV))
    far = cf.causal_conv1d(x, w, seq_offsets=torch.tensor([0, 12, 400], dtype=torch.int32, device=DEV))
    assert torch.equal(good, far)


def test_other_stream():
    """Work goes on the caller's stream: inputs made there just before the call, nothing synchronised between."""
    x, w = rnd((64, 256), 330, BF).to(DEV), torch.ones(256, dtype=BF, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y = (x.float() * 2).to(BF)
        q, s, _ = cf.rms_norm_q8(y, w)
        wq = torch.ones(32, 256, dtype=I8, device=DEV)
        out = cf.matmul_q8(q, s, wq, torch.ones(32, device=DEV), out_dtype=F32)
        z = cf.causal_conv1d(out, torch.ones(32, 2, device=DEV))
    side.synchronize()
    q0, s0, _ = cf.rms_norm_q8((x.float() * 2).to(BF), w)
    want = (q0.float().sum(1) * s0)[:, None].expand(64, 32)
    assert torch.allclose(out, want, rtol=1e-6)
    assert torch.allclose(z[1:], want[1:] + want[:-1], rtol=1e-5, atol=1e-5)


def test_graph_replays():
    """The mixer's calls captured into one graph; every replay equals the eager calls, with eager work between."""
    T, C = 130, 2 * 64 + 64
    x, r = rnd((T, 128), 340, BF).to(DEV), rnd((T, 128), 341, BF).to(DEV)
    nw = torch.ones(128, dtype=BF, device=DEV)
    wq, ws = eight((C, 128), 342, I8).to(DEV), (rnd(C, 343).abs() * 0.01).to(DEV)
    cw = rnd((C, 4), 344, BF).to(DEV)
    g, beta = -rnd((T, 1), 345).abs().to(DEV), torch.sigmoid(rnd((T, 1), 346)).to(DEV)
    fin = torch.zeros(1, 1, 64, 64, device=DEV)

    def step():
        q, s, h = cf.rms_norm_q8(x, nw, residual=r)
        y = cf.causal_conv1d(cf.matmul_q8(q, s, wq, ws), cw, activation="silu")
        o = cf.gated_delta_rule(y[:, :64].view(T, 1, 64), y[:, 64:128].view(T, 1, 64), y[:, 128:].view(T, 1, 64), g, beta,
                                normalize=True, final_state=fin)
        return h, o

    h0, o0 = (t.clone() for t in step())
    fin0 = fin.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, o = step()
    for _ in range(4):
        h.zero_(), o.zero_(), fin.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, h0) and torch.equal(o, o0) and torch.equal(fin, fin0)
        (x.float() @ x.float().t()).sum().item()
