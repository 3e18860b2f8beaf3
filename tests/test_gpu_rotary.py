"""Head norms with rotation on the GPU against their definition in 64 bits (scan_ref.py)."""
import pytest
import torch

import convolution_forward_amd as cf
import mixer_ref
import scan_ref as ref
from test_gpu_mixer import BF, DEV, F32, rnd

pytestmark = pytest.mark.gpu


def inputs(tokens, hq, hk, D, R, dtype, seed, far=0):
    q, k = rnd((tokens, hq, D), seed, dtype, 2.0), rnd((tokens, hk, D), seed + 1, dtype, 0.5)
    wq, wk = (rnd(D, seed + 2 + i) * 0.2 + 1 for i in (0, 1))
    pos = torch.randint(0, 5000, (tokens,), generator=torch.Generator().manual_seed(seed)) + far
    return q, k, wq.to(dtype), wk.to(dtype), pos, cf.rotary_frequencies(R, device="cpu")[0]


def check(got, x, pos, f, w, what, eps=1e-6, interleaved=False, scale=1.0):
    y, bound = ref.rotary(x, pos, f, w, eps, interleaved, scale)
    mixer_ref.check(got, y, bound, what, x.dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(2, 2), (3, 2), (6, 4), (24, 12), (33, 32), (64, 64), (64, 20), (80, 80), (80, 40), (128, 128),
                                 (128, 64), (128, 2), (160, 40), (256, 256), (256, 64), (260, 130), (512, 512), (511, 300)])
def test_heads(D, R, interleaved, dtype):
    for tokens, hq, hk, norm in ((1, 3, 1, True), (5, 2, 2, False), (130, 9, 3, True)):
        q, k, wq, wk, pos, f = inputs(tokens, hq, hk, D, R, dtype, D + R)
        gq, gk = cf.rotary(q.to(DEV), pos.to(DEV), f.to(DEV), k=k.to(DEV), q_weight=wq.to(DEV) if norm else None,
                           k_weight=wk.to(DEV) if norm else None, eps=1e-5, interleaved=interleaved, scale=1.25)
        check(gq, q, pos, f, wq if norm else None, "q", 1e-5, interleaved, 1.25)
        check(gk, k, pos, f, wk if norm else None, "k", 1e-5, interleaved, 1.25)


@pytest.mark.parametrize("tokens,hq,hk", [(1, 1, 0), (1, 64, 8), (3, 40, 8), (64, 16, 2), (1000, 5, 0), (2047, 2, 1)])
def test_tokens_and_heads(tokens, hq, hk):
    q, k, wq, wk, pos, f = inputs(tokens, hq, max(hk, 1), 128, 128, BF, tokens)
    got = cf.rotary(q.to(DEV), pos.int().to(DEV), f.to(DEV), k=k.to(DEV) if hk else None, q_weight=wq.to(DEV))
    check(got[0] if hk else got, q, pos, f, wq, "q")
    if hk:
        check(got[1], k, pos, f, None, "k")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_positions(dtype):
    """Far, negative and equal positions, and frequencies that are negative, zero or above one turn a position."""
    pos = torch.tensor([0, -1, 7, 7, 1000003, 2 ** 24 + 1, -(2 ** 31), 2 ** 31 - 1, 2 ** 33 + 5, 123456789])
    f = torch.tensor([1.0, -0.3, 0.0, 8.0, 1e-5, 0.7320508, 3.1415927, 1e-30])
    q = rnd((10, 2, 16), 5, dtype)
    check(cf.rotary(q.to(DEV), pos.to(DEV), f.to(DEV)), q, pos, f, None, "int64")
    near = pos.clamp(-(2 ** 31), 2 ** 31 - 1)
    check(cf.rotary(q.to(DEV), near.int().to(DEV), f.to(DEV), interleaved=True), q, near, f, None, "int32", interleaved=True)


@pytest.mark.parametrize("shift", [0, 1, 4])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place_in_one_buffer(dtype, shift):
    """Queries and keys as columns of a row, rotated where they are; the values beside them stay."""
    t, hq, hk, D = 37, 4, 2, 64
    row = (hq + 2 * hk) * D + 8
    buf = rnd(t * row + shift, 6, dtype).to(DEV)
    rows = buf[shift:].view(t, row)
    before = rows.cpu().clone()
    q, k = (rows[:, i * D:j * D].unflatten(-1, (-1, D)) for i, j in ((0, hq), (hq, hq + hk)))
    wq, pos, f = rnd(D, 7, dtype), torch.arange(t) * 3, cf.rotary_frequencies(D, device="cpu")[0]
    got = cf.rotary(q, pos.to(DEV), f.to(DEV), k=k, q_weight=wq.to(DEV), out=q, k_out=k)
    assert got[0].data_ptr() == q.data_ptr() and got[1].data_ptr() == k.data_ptr()
    check(q, before[:, :hq * D].view(t, hq, D), pos, f, wq, "q")
    check(k, before[:, hq * D:(hq + hk) * D].view(t, hk, D), pos, f, None, "k")
    assert torch.equal(rows[:, (hq + hk) * D:].cpu(), before[:, (hq + hk) * D:])


def test_layouts():
    """Heads outside tokens, a batch axis, heads at a pitch, and outputs with a pitch of their own."""
    t, h, D = 12, 3, 32
    x, pos, f = rnd((h, t, D), 8, BF), torch.arange(t), cf.rotary_frequencies(D, device="cpu")[0]
    got = cf.rotary(x.to(DEV).transpose(0, 1), pos.to(DEV), f.to(DEV))
    check(got, x.transpose(0, 1), pos, f, None, "heads outside")
    four = cf.rotary(x.transpose(0, 1).reshape(3, 4, h, D).to(DEV), pos.to(DEV), f.to(DEV))
    assert four.shape == (3, 4, h, D) and torch.equal(four.view(t, h, D), got)
    out = torch.full((t, h, D + 5), 7.0, dtype=BF, device=DEV)
    cf.rotary(x.to(DEV).transpose(0, 1), pos.to(DEV), f.to(DEV), out=out[..., :D])
    assert torch.equal(out[..., :D], got) and (out[..., D:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_special_heads(dtype):
    """Zeros and tiny heads without an eps, squares past fp32's range, and values that are not finite in one head only."""
    q = rnd((8, 2, 64), 9, dtype)
    q[0, 0] = 0
    q[1, 0] = -0.0
    q[2] *= 1e-25
    q[3] *= 1e30
    q[4, 0] = 0
    q[4, 0, 63] = -1e-38
    w, pos, f = rnd(64, 10, dtype), torch.arange(8), cf.rotary_frequencies(32, device="cpu")[0]
    check(cf.rotary(q.to(DEV), pos.to(DEV), f.to(DEV), q_weight=w.to(DEV), eps=0.0), q, pos, f, w, "eps 0", eps=0.0)
    q[6, 1, 40] = float("nan")
    q[7, 0, 5] = float("inf")
    got = cf.rotary(q.to(DEV), pos.to(DEV), f.to(DEV), q_weight=w.to(DEV)).cpu()
    assert torch.isnan(got[6, 1]).all() and torch.isnan(got[7, 0, 5])
    ok = torch.ones(8, 2, dtype=torch.bool)
    ok[6, 1] = ok[7, 0] = False
    want, bound = ref.rotary(q, pos, f, w, 1e-6, False, 1.0)
    mixer_ref.check(got[ok], want[ok], bound[ok], "others", dtype)
    got = cf.rotary(q.to(DEV), pos.to(DEV), f.to(DEV)).cpu()
    assert torch.isnan(got[6, 1, 40]) and torch.isfinite(got[6, 1, :40]).all() and torch.isfinite(got[7, 0, 32:]).all()
    bad = f.clone()
    bad[3] = float("inf")
    got = cf.rotary(q[:5].to(DEV), pos[:5].to(DEV), bad.to(DEV)).cpu()
    assert torch.isnan(got[..., [3, 19]]).all() and torch.isfinite(got[..., [2, 4, 18, 20, 40]]).all()


def test_no_tokens():
    q, k = cf.rotary(torch.empty(0, 2, 64, dtype=BF, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV),
                     torch.ones(32, device=DEV), k=torch.empty(0, 1, 64, dtype=BF, device=DEV))
    assert q.shape == (0, 2, 64) and k.shape == (0, 1, 64)


def test_refusals():
    q, k = torch.zeros(4, 2, 64, device=DEV), torch.zeros(4, 1, 64, device=DEV)
    pos, f, w = torch.arange(4, device=DEV), torch.ones(16, device=DEV), torch.ones(64, device=DEV)
    for kw in (dict(k=k[:3]), dict(k=k.bfloat16()), dict(q_weight=w.bfloat16()), dict(q_weight=w[:32]), dict(k_weight=w),
               dict(k_out=k), dict(positions=pos.float()), dict(positions=pos[:3]), dict(positions=pos.expand(2, 4)),
               dict(frequencies=f.double()), dict(frequencies=torch.ones(33, device=DEV)), dict(frequencies=f[::2]),
               dict(out=q.bfloat16()), dict(out=q[:, :1]), dict(q=q.transpose(1, 2)), dict(q=q[0]), dict(q=q.half()),
               dict(positions=pos.cpu()), dict(out=q.flatten()[64:448].view(3, 2, 64)),
               dict(q=torch.zeros(4, 2, 513, device=DEV))):
        with pytest.raises(ValueError):
            cf.rotary(**{**dict(q=q, positions=pos, frequencies=f), **kw})


def test_many_heads_and_tokens():
    """More tokens than a few workgroups take: the same as the call on some of them."""
    t = 70001
    q = torch.arange(t * 2 * 64, device=DEV).remainder(8191).sub(4000).to(BF).view(t, 2, 64)
    pos, f, w = torch.arange(t, device=DEV), cf.rotary_frequencies(64)[0], rnd(64, 12, BF).to(DEV)
    got = cf.rotary(q, pos, f, q_weight=w)
    for some in (slice(0, 5), slice(34000, 34100), slice(t - 3, t)):
        assert torch.equal(got[some], cf.rotary(q[some], pos[some], f, q_weight=w))
    h = 70000
    q = q.view(-1)[:2 * h * 8].view(2, h, 8)[:, :65535]
    got = cf.rotary(q, pos[:2], f[:4])
    assert torch.equal(got[:, 60000:60010], cf.rotary(q[:, 60000:60010], pos[:2], f[:4]))
