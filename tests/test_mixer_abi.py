"""Refusals of the token-mixer calls, on the host: every argument error is returned before any HIP call (fake, distinct
device addresses, never dereferenced). And the 64-bit definitions used by the GPU tests, checked on small numbers."""
import ctypes

import pytest
import torch

import convolution_forward_amd as cf
import mixer_ref as ref

P = [0x10000000000 + i * 0x1000000000 for i in range(16)]      # far apart: no two tensors meet


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(cf.LIB_PATH):
        from convolution_forward_amd import build
        build.build()
    return cf.load_library()


def strides(*v):
    return (ctypes.c_int64 * len(v))(*v)


NORM = dict(x=P[0], xs=64, r=P[1], rs=64, w=P[2], h=P[3], hs=64, q=P[4], qs=64, scale=P[5], rows=4, width=64, eps=1e-6,
            dt=cf.CONV_BF16, qdt=cf.CONV_I8, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), cf.CONV_ERR_NULL), (dict(w=None), cf.CONV_ERR_NULL), (dict(q=None), cf.CONV_ERR_NULL),
    (dict(scale=None), cf.CONV_ERR_NULL), (dict(h=None), cf.CONV_ERR_NULL),
    (dict(r=None, rs=0), cf.CONV_ERR_UNSUPPORTED),                      # a sum without a residual
    (dict(rows=-1), cf.CONV_ERR_NONPOSITIVE), (dict(width=0), cf.CONV_ERR_NONPOSITIVE),
    (dict(dt=cf.CONV_I8), cf.CONV_ERR_DTYPE), (dict(qdt=cf.CONV_BF16), cf.CONV_ERR_DTYPE), (dict(qdt=9), cf.CONV_ERR_DTYPE),
    (dict(xs=63), cf.CONV_ERR_LAYOUT), (dict(rs=63), cf.CONV_ERR_LAYOUT), (dict(hs=1), cf.CONV_ERR_LAYOUT),
    (dict(qs=0), cf.CONV_ERR_LAYOUT), (dict(x=P[0] + 1), cf.CONV_ERR_LAYOUT), (dict(scale=P[5] + 2), cf.CONV_ERR_LAYOUT),
    (dict(xs=1 << 60), cf.CONV_ERR_LAYOUT),
    (dict(q=P[0]), cf.CONV_ERR_ALIAS), (dict(q=P[2]), cf.CONV_ERR_ALIAS), (dict(scale=P[4]), cf.CONV_ERR_ALIAS),
    (dict(h=P[0] + 128), cf.CONV_ERR_ALIAS), (dict(h=P[1], hs=65), cf.CONV_ERR_ALIAS), (dict(h=P[2]), cf.CONV_ERR_ALIAS),
    (dict(scale=P[0]), cf.CONV_ERR_ALIAS),
])
def test_norm_refusals(lib, change, status):
    assert lib.conv_rms_norm_q8_fwd(*{**NORM, **change}.values()) == status


def test_norm_of_no_rows(lib):
    assert lib.conv_rms_norm_q8_fwd(*{**NORM, "rows": 0}.values()) == cf.CONV_OK


PRODUCT = dict(x=P[0], xs=64, sx=P[1], w=P[2], ws=64, sw=P[3], b=P[4], y=P[5], ys=32, M=4, N=32, K=64, q=cf.CONV_I8,
               yd=cf.CONV_BF16, variant=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), cf.CONV_ERR_NULL), (dict(w=None), cf.CONV_ERR_NULL), (dict(sx=None), cf.CONV_ERR_NULL),
    (dict(sw=None), cf.CONV_ERR_NULL), (dict(y=None), cf.CONV_ERR_NULL),
    (dict(M=-1), cf.CONV_ERR_NONPOSITIVE), (dict(N=0), cf.CONV_ERR_NONPOSITIVE), (dict(K=0), cf.CONV_ERR_NONPOSITIVE),
    (dict(q=cf.CONV_F32), cf.CONV_ERR_DTYPE), (dict(yd=cf.CONV_I8), cf.CONV_ERR_DTYPE),
    (dict(K=131072, xs=131072, ws=131072), cf.CONV_ERR_UNSUPPORTED), (dict(variant=7), cf.CONV_ERR_UNSUPPORTED),
    (dict(xs=63), cf.CONV_ERR_LAYOUT), (dict(ws=63), cf.CONV_ERR_LAYOUT), (dict(ys=31), cf.CONV_ERR_LAYOUT),
    (dict(sx=P[1] + 1), cf.CONV_ERR_LAYOUT), (dict(y=P[5] + 1), cf.CONV_ERR_LAYOUT), (dict(b=P[4] + 2), cf.CONV_ERR_LAYOUT),
    (dict(y=P[0]), cf.CONV_ERR_ALIAS), (dict(y=P[2] + 64), cf.CONV_ERR_ALIAS), (dict(y=P[1]), cf.CONV_ERR_ALIAS),
    (dict(y=P[4] + 64), cf.CONV_ERR_ALIAS),
])
def test_product_refusals(lib, change, status):
    assert lib.conv_matmul_q8_fwd(*{**PRODUCT, **change}.values()) == status


CONV = dict(x=P[0], xs=32, w=P[1], b=P[2], y=P[3], ys=32, off=P[4], si=P[5], so=P[6], slots=P[7], num=4, T=20, n=3, C=32,
            taps=4, silu=1, dt=cf.CONV_BF16, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), cf.CONV_ERR_NULL), (dict(w=None), cf.CONV_ERR_NULL), (dict(y=None), cf.CONV_ERR_NULL),
    (dict(C=0), cf.CONV_ERR_NONPOSITIVE), (dict(T=-1), cf.CONV_ERR_NONPOSITIVE), (dict(n=0), cf.CONV_ERR_NONPOSITIVE),
    (dict(num=0), cf.CONV_ERR_NONPOSITIVE), (dict(dt=cf.CONV_I8), cf.CONV_ERR_DTYPE),
    (dict(taps=1), cf.CONV_ERR_UNSUPPORTED), (dict(taps=9), cf.CONV_ERR_UNSUPPORTED),
    (dict(off=None), cf.CONV_ERR_SHAPE),                                # 20 tokens are not 3 equal sequences
    (dict(slots=None, num=2), cf.CONV_ERR_SHAPE),
    (dict(xs=31), cf.CONV_ERR_LAYOUT), (dict(ys=31), cf.CONV_ERR_LAYOUT), (dict(x=P[0] + 1), cf.CONV_ERR_LAYOUT),
    (dict(off=P[4] + 2), cf.CONV_ERR_LAYOUT), (dict(so=P[6] + 1), cf.CONV_ERR_LAYOUT),
    (dict(y=P[0]), cf.CONV_ERR_ALIAS), (dict(y=P[5]), cf.CONV_ERR_ALIAS), (dict(so=P[5] + 64), cf.CONV_ERR_ALIAS),
    (dict(so=P[0]), cf.CONV_ERR_ALIAS), (dict(so=P[3]), cf.CONV_ERR_ALIAS), (dict(so=P[4]), cf.CONV_ERR_ALIAS),
])
def test_conv_refusals(lib, change, status):
    assert lib.conv_causal1d_fwd(*{**CONV, **change}.values()) == status


DELTA = dict(q=P[0], qs=None, k=P[1], ks=None, v=P[2], vs=None, g=P[3], beta=P[4], off=P[5], si=P[6], so=P[7], slots=P[8],
             num=4, o=P[9], os=None, ws=P[10], wsb=1 << 34, T=200, n=3, Hk=2, Hv=4, Dk=64, Dv=32, scale=0.1, norm=1,
             dt=cf.CONV_BF16, variant=0, stream=None)


@pytest.mark.parametrize("change,status", [
    *[({name: None}, cf.CONV_ERR_NULL) for name in ("q", "k", "v", "g", "beta", "o")],
    *[({name: 0}, cf.CONV_ERR_NONPOSITIVE) for name in ("n", "Hk", "Hv", "Dk", "Dv", "num")],
    (dict(T=-1), cf.CONV_ERR_NONPOSITIVE), (dict(Hv=3), cf.CONV_ERR_SHAPE), (dict(off=None), cf.CONV_ERR_SHAPE),
    (dict(slots=None, num=2), cf.CONV_ERR_SHAPE), (dict(dt=cf.CONV_E4M3), cf.CONV_ERR_DTYPE),
    (dict(Dk=257), cf.CONV_ERR_UNSUPPORTED), (dict(variant=5), cf.CONV_ERR_UNSUPPORTED),
    (dict(qs=strides(-1, 64)), cf.CONV_ERR_LAYOUT), (dict(os=strides(31, 32)), cf.CONV_ERR_LAYOUT),
    (dict(os=strides(128, 16)), cf.CONV_ERR_LAYOUT), (dict(q=P[0] + 1), cf.CONV_ERR_LAYOUT),
    (dict(g=P[3] + 2), cf.CONV_ERR_LAYOUT), (dict(ws=P[10] + 8), cf.CONV_ERR_LAYOUT),
    (dict(vs=strides(1 << 40, 1 << 40), T=1 << 29, off=P[5]), cf.CONV_ERR_LAYOUT),
    (dict(o=P[2]), cf.CONV_ERR_ALIAS), (dict(o=P[6] + 64), cf.CONV_ERR_ALIAS), (dict(so=P[6] + 4), cf.CONV_ERR_ALIAS),
    (dict(so=P[0]), cf.CONV_ERR_ALIAS), (dict(so=P[9]), cf.CONV_ERR_ALIAS), (dict(so=P[8]), cf.CONV_ERR_ALIAS),
])
def test_delta_refusals(lib, change, status):
    assert lib.conv_delta_rule_fwd(*{**DELTA, **change}.values()) == status


def test_delta_workspace_query(lib):
    assert cf.delta_rule_workspace(1, 1, 16, 32, 128, 128) >= 0
    assert cf.delta_rule_workspace(0, 1, 1, 1, 64, 64) >= 0
    assert cf.delta_rule_workspace(1, 1, 2, 3, 64, 64) == -1
    assert cf.delta_rule_workspace(1, 1, 1, 1, 300, 64) == -1
    # More heads and sequences than a grid of chunks holds: token by token, without a workspace.
    assert cf.delta_rule_workspace(40000 * 64, 40000, 16, 32, 128, 128) == 0
    assert cf.delta_rule_workspace(40000 * 64, 40000, 16, 32, 128, 128, variant=cf.VARIANT_TILED) == -1


def test_binding_rejects_cpu_tensors(lib):
    x = torch.zeros(2, 16)
    for call in (lambda: cf.rms_norm_q8(x, torch.ones(16)),
                 lambda: cf.matmul_q8(x.to(torch.int8), x[:, 0], x.to(torch.int8), x[:, 0]),
                 lambda: cf.causal_conv1d(x, torch.ones(16, 2)),
                 lambda: cf.gated_delta_rule(x.view(2, 1, 16), x.view(2, 1, 16), x.view(2, 1, 16), x[:, :1], x[:, :1])):
        with pytest.raises(ValueError, match="GPU"):
            call()


# ---- the definitions themselves --------------------------------------------------------------------------------------


def test_delta_definition_on_small_numbers():
    """One key direction: the state's column for it moves to v by beta, and is read back by the same direction."""
    one = torch.tensor([[[1.0, 0.0]]] * 3)
    v = torch.tensor([[[4.0]], [[2.0]], [[0.0]]])
    g = torch.tensor([[0.0], [0.0], [-0.6931471805599453]])
    beta = torch.tensor([[1.0], [0.5], [0.0]])
    o, _, s, _ = ref.delta(one, one, v, g, beta, 1.0, False, [3], None)
    assert torch.allclose(o.flatten(), torch.tensor([4.0, 3.0, 1.5], dtype=torch.float64), rtol=1e-6)
    assert torch.allclose(s.flatten(), torch.tensor([1.5, 0.0], dtype=torch.float64), rtol=1e-6)


def test_conv_definition_against_the_oracle(oracle_mod):
    """The causal convolution is the depthwise operator with its padding before the signal only."""
    x, w = torch.randn(12, 5), torch.randn(5, 4)
    y, _, new = ref.conv(x, w, None, False, [12], None)
    planes = torch.cat([torch.zeros(3, 5), x]).t().contiguous().view(1, 5, 1, 15)
    want = oracle_mod.depthwise_nchw(planes, w.view(5, 1, 4), mode="fast")
    assert torch.allclose(y.float(), torch.from_numpy(want).view(5, 12).t(), atol=1e-5)
    assert torch.equal(new[0].float(), x[9:])


def test_norm_definition_on_small_numbers():
    h, y, _ = ref.norm(torch.tensor([[3.0, 4.0]]), torch.tensor([1.0, 2.0]), torch.tensor([[0.0, 0.0]]), 0.0)
    r = (12.5) ** 0.5
    assert torch.allclose(y, torch.tensor([[3 / r, 8 / r]], dtype=torch.float64))
    assert torch.equal(h, torch.tensor([[3.0, 4.0]]))


def test_bounds_reject_a_planted_mistake():
    """A dropped decay, a swapped head or a tap too late is far outside the bounds."""
    gen = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(40, 2, 16, generator=gen) for _ in range(3))
    g, beta = -torch.rand(40, 2, generator=gen), torch.rand(40, 2, generator=gen)
    o, bo, _, _ = ref.delta(q, k, v, g, beta, 1.0, True, [40], None)
    wrong, _, _, _ = ref.delta(q, k, v, 0.999 * g, beta, 1.0, True, [40], None)
    swapped, _, _, _ = ref.delta(q.flip(1), k, v, g, beta, 1.0, True, [40], None)
    for bad in (wrong, swapped):
        with pytest.raises(AssertionError):
            ref.check(bad.float(), o, bo, "o")
    ref.check(o.float(), o, bo, "o")
