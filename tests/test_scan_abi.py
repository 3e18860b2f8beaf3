"""Refusals of the rotary and selective scan calls, on the host: every argument error is returned before any HIP call
(fake, distinct device addresses, never dereferenced). And the 64-bit definitions that the GPU tests use, on small numbers."""
import math

import pytest
import torch

import convolution_forward_amd as cf
import scan_ref as ref
from mixer_ref import U
from test_mixer_abi import P, lib, strides  # noqa: F401

F32, BF = torch.float32, torch.bfloat16

ROTARY = dict(q=P[0], qs=None, k=P[1], ks=None, pos=P[2], bits=64, f=P[3], qw=P[4], kw=P[5], qo=P[6], qos=None, ko=P[7],
              kos=None, T=5, Hq=4, Hk=2, D=64, R=32, eps=1e-6, scale=1.0, inter=0, dt=cf.CONV_BF16, stream=None)


@pytest.mark.parametrize("change,status", [
    *[({name: None}, cf.CONV_ERR_NULL) for name in ("q", "k", "pos", "f", "qo", "ko")],
    (dict(T=-1), cf.CONV_ERR_NONPOSITIVE), (dict(Hq=0), cf.CONV_ERR_NONPOSITIVE), (dict(Hk=-1), cf.CONV_ERR_NONPOSITIVE),
    (dict(D=0), cf.CONV_ERR_NONPOSITIVE), (dict(R=0), cf.CONV_ERR_NONPOSITIVE),
    (dict(R=31), cf.CONV_ERR_SHAPE), (dict(R=66), cf.CONV_ERR_SHAPE), (dict(dt=cf.CONV_I8), cf.CONV_ERR_DTYPE),
    (dict(bits=16), cf.CONV_ERR_UNSUPPORTED), (dict(D=514), cf.CONV_ERR_UNSUPPORTED),
    (dict(T=1 << 24), cf.CONV_ERR_UNSUPPORTED), (dict(Hq=65536), cf.CONV_ERR_UNSUPPORTED),
    (dict(q=P[0] + 1), cf.CONV_ERR_LAYOUT), (dict(ko=P[7] + 1), cf.CONV_ERR_LAYOUT), (dict(pos=P[2] + 4), cf.CONV_ERR_LAYOUT),
    (dict(f=P[3] + 2), cf.CONV_ERR_LAYOUT), (dict(kw=P[5] + 1), cf.CONV_ERR_LAYOUT),
    (dict(qs=strides(-1, 64)), cf.CONV_ERR_LAYOUT), (dict(qos=strides(64, 64)), cf.CONV_ERR_LAYOUT),
    (dict(kos=strides(128, 32)), cf.CONV_ERR_LAYOUT), (dict(qs=strides(1 << 41, 64)), cf.CONV_ERR_LAYOUT),
    (dict(qo=P[0] + 128), cf.CONV_ERR_ALIAS), (dict(qo=P[0], qos=strides(512, 64)), cf.CONV_ERR_ALIAS),
    (dict(qo=P[1]), cf.CONV_ERR_ALIAS), (dict(ko=P[0]), cf.CONV_ERR_ALIAS), (dict(ko=P[6]), cf.CONV_ERR_ALIAS),
    (dict(qo=P[2]), cf.CONV_ERR_ALIAS), (dict(ko=P[3]), cf.CONV_ERR_ALIAS), (dict(ko=P[4]), cf.CONV_ERR_ALIAS),
    (dict(qo=P[5]), cf.CONV_ERR_ALIAS),
    # q and k as columns of one buffer of rows, overwritten: k's columns begin inside q's.
    (dict(qs=strides(384, 64), qo=P[0], qos=strides(384, 64), k=P[0] + 500, ks=strides(384, 64)), cf.CONV_ERR_ALIAS),
    (dict(qs=strides(384, 64), qo=P[0], qos=strides(384, 64), k=P[0] + 520, ks=strides(384, 64)), cf.CONV_ERR_ALIAS),
])
def test_rotary_refusals(lib, change, status):  # noqa: F811
    assert lib.conv_rotary_fwd(*{**ROTARY, **change}.values()) == status


def test_rotary_without_tokens_or_keys(lib):  # noqa: F811
    assert lib.conv_rotary_fwd(*{**ROTARY, "T": 0}.values()) == cf.CONV_OK
    assert lib.conv_rotary_fwd(*{**ROTARY, "T": 0, "Hk": 0, "k": None, "ko": None}.values()) == cf.CONV_OK


SCAN = dict(x=P[0], xs=32, d=P[1], ds=32, a=P[2], b=P[3], bs=None, c=P[4], cs=None, skip=P[5], g=P[6], gs=32, bias=P[7],
            y=P[8], ys=32, off=P[9], si=P[10], so=P[11], slots=P[12], num=4, ws=P[13], wsb=1 << 34, T=20, n=3, C=32, G=2,
            N=16, soft=1, dt=cf.CONV_BF16, variant=0, stream=None)


@pytest.mark.parametrize("change,status", [
    *[({name: None}, cf.CONV_ERR_NULL) for name in ("x", "d", "a", "b", "c", "y")],
    *[({name: 0}, cf.CONV_ERR_NONPOSITIVE) for name in ("n", "C", "G", "N", "num")],
    (dict(T=-1), cf.CONV_ERR_NONPOSITIVE), (dict(G=3), cf.CONV_ERR_SHAPE), (dict(off=None), cf.CONV_ERR_SHAPE),
    (dict(slots=None, num=2), cf.CONV_ERR_SHAPE), (dict(dt=cf.CONV_I8), cf.CONV_ERR_DTYPE),
    (dict(N=257), cf.CONV_ERR_UNSUPPORTED), (dict(variant=5), cf.CONV_ERR_UNSUPPORTED),
    (dict(xs=31), cf.CONV_ERR_LAYOUT), (dict(ds=31), cf.CONV_ERR_LAYOUT), (dict(gs=31), cf.CONV_ERR_LAYOUT),
    (dict(ys=31), cf.CONV_ERR_LAYOUT), (dict(bs=strides(-1, 16)), cf.CONV_ERR_LAYOUT), (dict(x=P[0] + 1), cf.CONV_ERR_LAYOUT),
    (dict(a=P[2] + 2), cf.CONV_ERR_LAYOUT), (dict(ws=P[13] + 8), cf.CONV_ERR_LAYOUT), (dict(so=P[11] + 2), cf.CONV_ERR_LAYOUT),
    (dict(off=P[9] + 2), cf.CONV_ERR_LAYOUT),
    (dict(y=P[0]), cf.CONV_ERR_ALIAS), (dict(y=P[6]), cf.CONV_ERR_ALIAS), (dict(y=P[10]), cf.CONV_ERR_ALIAS),
    (dict(so=P[10] + 64), cf.CONV_ERR_ALIAS), (dict(so=P[2]), cf.CONV_ERR_ALIAS), (dict(so=P[8]), cf.CONV_ERR_ALIAS),
    (dict(so=P[12]), cf.CONV_ERR_ALIAS),
])
def test_scan_refusals(lib, change, status):  # noqa: F811
    assert lib.conv_selective_scan_fwd(*{**SCAN, **change}.values()) == status


HEADS = dict(x=P[0], xs=None, d=P[1], ds=4, a=P[2], b=P[3], bs=None, c=P[4], cs=None, skip=P[5], g=P[6], gs=None, bias=P[7],
             y=P[8], ys=None, off=P[9], si=P[10], so=P[11], slots=P[12], num=4, ws=P[13], wsb=1 << 34, T=200, n=3, H=4, P=32,
             G=2, N=64, soft=1, dt=cf.CONV_BF16, variant=0, stream=None)


@pytest.mark.parametrize("change,status", [
    *[({name: None}, cf.CONV_ERR_NULL) for name in ("x", "d", "a", "b", "c", "y")],
    *[({name: 0}, cf.CONV_ERR_NONPOSITIVE) for name in ("n", "H", "P", "G", "N", "num")],
    (dict(T=-1), cf.CONV_ERR_NONPOSITIVE), (dict(G=3), cf.CONV_ERR_SHAPE), (dict(off=None), cf.CONV_ERR_SHAPE),
    (dict(slots=None, num=2), cf.CONV_ERR_SHAPE), (dict(dt=cf.CONV_E4M3), cf.CONV_ERR_DTYPE),
    (dict(N=257), cf.CONV_ERR_UNSUPPORTED), (dict(variant=5), cf.CONV_ERR_UNSUPPORTED),
    (dict(ds=3), cf.CONV_ERR_LAYOUT), (dict(xs=strides(-1, 32)), cf.CONV_ERR_LAYOUT), (dict(ys=strides(31, 32)), cf.CONV_ERR_LAYOUT),
    (dict(ys=strides(128, 16)), cf.CONV_ERR_LAYOUT), (dict(x=P[0] + 1), cf.CONV_ERR_LAYOUT), (dict(a=P[2] + 2), cf.CONV_ERR_LAYOUT),
    (dict(ws=P[13] + 8), cf.CONV_ERR_LAYOUT), (dict(gs=strides(1 << 41, 32)), cf.CONV_ERR_LAYOUT),
    (dict(y=P[0]), cf.CONV_ERR_ALIAS), (dict(y=P[6]), cf.CONV_ERR_ALIAS), (dict(y=P[10]), cf.CONV_ERR_ALIAS),
    (dict(so=P[10] + 64), cf.CONV_ERR_ALIAS), (dict(so=P[2]), cf.CONV_ERR_ALIAS), (dict(so=P[8]), cf.CONV_ERR_ALIAS),
    (dict(so=P[12]), cf.CONV_ERR_ALIAS),
])
def test_heads_refusals(lib, change, status):  # noqa: F811
    assert lib.conv_selective_scan_heads_fwd(*{**HEADS, **change}.values()) == status


def test_workspace_queries(lib):  # noqa: F811
    assert cf.selective_scan_workspace(1, 1, 64, 1, 16) >= 0 and cf.selective_scan_workspace(0, 1, 64, 1, 16) >= 0
    assert cf.selective_scan_workspace(1, 1, 64, 3, 16) == -1 and cf.selective_scan_workspace(1, 1, 64, 1, 300) == -1
    assert cf.selective_scan_heads_workspace(1, 1, 4, 64, 2, 128) >= 0
    assert cf.selective_scan_heads_workspace(1, 1, 4, 64, 3, 128) == -1
    with pytest.raises(ValueError):
        cf.selective_scan_workspace(1, 1, 64, 1, 16, dtype=torch.float16)


def test_tensors_on_the_host_are_refused():
    x, a, b = torch.zeros(4, 8), torch.zeros(8, 4), torch.zeros(4, 1, 4)
    with pytest.raises(ValueError, match="GPU"):
        cf.selective_scan(x, x, a, b, b)
    with pytest.raises(ValueError, match="GPU"):
        cf.selective_scan_heads(x[:, None], x[:, :1], a[0], b, b)
    with pytest.raises(ValueError, match="GPU"):
        cf.rotary(x[:, None], torch.arange(4), torch.ones(4))
    with pytest.raises(ValueError, match="tensor"):
        cf.rotary([1.0], torch.arange(4), torch.ones(4))


# ---- frequencies -----------------------------------------------------------------------------------------------------


def test_frequencies():
    f, scale = cf.rotary_frequencies(8, base=10000.0, device="cpu")
    assert scale == 1.0 and f.dtype == F32
    assert torch.equal(f, torch.tensor([1.0, 0.1, 0.01, 0.001]))
    assert torch.equal(cf.rotary_frequencies(8, scaling="linear", factor=4.0, device="cpu")[0], f / 4)
    g, _ = cf.rotary_frequencies(8, scaling="base", factor=8.0, device="cpu")
    assert g[0] == 1.0 and math.isclose(g[-1], 0.001 / 8, rel_tol=1e-6)
    for kind in ("parts", "wavelength"):
        g, scale = cf.rotary_frequencies(128, scaling=kind, factor=16.0, trained=4096, fast=32.0, slow=1.0, device="cpu")
        f, _ = cf.rotary_frequencies(128, device="cpu")
        turns = 4096 * f.double() / (2 * math.pi)
        assert scale == (0.1 * math.log(16.0) + 1.0 if kind == "parts" else 1.0)
        # By index the ramp ends within one index of the bounds.
        sure_fast, sure_slow = turns >= 32.0 * 1.16, turns <= 1.0 / 1.16
        assert torch.equal(g[sure_fast], f[sure_fast])
        assert torch.allclose(g[sure_slow], f[sure_slow] / 16, rtol=2 * U, atol=0)
        part = ((f / g - 1) / 15)
        assert (part[1:] >= part[:-1] - 1e-6).all() and 0.0 < part[(turns < 16) & (turns > 2)].min() < 1.0
        if kind == "wavelength":
            mid = (turns < 31) & (turns > 1.1)
            keep = (turns[mid] - 1) / 31
            assert torch.allclose(g[mid].double(), f[mid].double() * (keep + (1 - keep) / 16), rtol=4 * U, atol=0)


@pytest.mark.parametrize("args", [dict(rotated=0), dict(rotated=7), dict(rotated=8, scaling="other"), dict(rotated=8, base=1.0),
                                  dict(rotated=8, scaling="linear", factor=0.5), dict(rotated=8, scaling="parts", factor=2.0),
                                  dict(rotated=8, scaling="wavelength", factor=2.0, trained=100, fast=1.0, slow=1.0)])
def test_frequencies_refusals(args):
    with pytest.raises(ValueError):
        cf.rotary_frequencies(**{"device": "cpu", **args})


# ---- the definitions -------------------------------------------------------------------------------------------------


def test_rotary_definition():
    x = torch.tensor([[[3.0, 4.0, 1.0, 2.0, 5.0]]])
    quarter = torch.tensor([math.pi / 2, math.pi], dtype=F32)
    y, bound = ref.rotary(x, torch.tensor([1]), quarter, None, 0.0, False, 2.0)
    assert torch.allclose(y, torch.tensor([[[-2.0, -8.0, 6.0, -4.0, 5.0]]], dtype=torch.float64), atol=1e-6)
    y, _ = ref.rotary(x, torch.tensor([1]), quarter, None, 0.0, True, 1.0)
    assert torch.allclose(y, torch.tensor([[[-4.0, 3.0, -1.0, -2.0, 5.0]]], dtype=torch.float64), atol=1e-6)
    y, _ = ref.rotary(x, torch.tensor([0]), quarter, torch.full((5,), 2.0), 0.0, True, 1.0)
    assert torch.allclose(y, 2 * x.double() / math.sqrt(11.0))
    assert (bound >= 0).all() and bound.max() < 1e-5


def test_scan_definition():
    """Two tokens by hand, and the head form against the channel form with the same decay."""
    one = torch.ones(2, 1)
    a, half = torch.tensor([[-1.0]]), torch.tensor([[[0.5]], [[2.0]]])
    y, bound, h, bh = ref.channels(torch.tensor([[2.0], [3.0]]), one, a, half, one[:, None], torch.tensor([10.0]), None, None,
                                   False, [2], torch.tensor([[[4.0]]]))
    e = math.exp(-1.0)
    want = [4 * e + 1, (4 * e + 1) * e + 6]
    assert torch.allclose(y[:, 0], torch.tensor([want[0] + 20, want[1] + 30], dtype=torch.float64))
    assert math.isclose(h.item(), want[1]) and bound.max() < 1e-4 and bh.max() < 1e-4
    gen = torch.Generator().manual_seed(1)
    x, dt, b, c = (torch.randn(9, *s, generator=gen) for s in ((2, 3), (2,), (1, 4), (1, 4)))
    rate, gate, skip, bias = -torch.rand(2, generator=gen), torch.randn(9, 2, 3, generator=gen), torch.ones(2), torch.zeros(2)
    y1, _, h1, _ = ref.heads(x, dt, rate, b, c, skip, gate, bias, True, [5, 0, 4], None)
    wide = [t.repeat_interleave(3, -1) for t in (dt, rate, skip, bias)]
    y2, _, h2, _ = ref.channels(x.flatten(1), wide[0], wide[1][:, None].expand(6, 4), b, c, wide[2], gate.flatten(1), wide[3],
                                True, [5, 0, 4], None)
    assert torch.allclose(y1.flatten(1), y2) and torch.allclose(h1.flatten(1, 2), h2) and (h1[1] == 0).all()
