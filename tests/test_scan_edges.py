"""Limits of the selective scan calls on the host: sizes past a grid are refused, never cut."""
import pytest

import convolution_forward_amd as cf
from test_mixer_abi import lib  # noqa: F401  (fake addresses: nothing may be launched)
from test_scan_abi import HEADS, SCAN

AUTO, DIRECT, TILED = cf.VARIANT_AUTO, cf.VARIANT_DIRECT, cf.VARIANT_TILED
EQUAL = dict(off=None, slots=None, si=None, so=None)


@pytest.mark.parametrize("change", [
    dict(variant=DIRECT, T=1 << 24, n=1 << 24, C=64, xs=64, ds=64, gs=64, ys=64),           # a wave takes 16 channels
    dict(variant=AUTO, T=1 << 24, n=1 << 24, C=64, xs=64, ds=64, gs=64, ys=64),
    dict(variant=TILED, T=1 << 20, n=1 << 20, C=1024, G=1, xs=1024, ds=1024, gs=1024, ys=1024),   # 2^26 workgroups
    dict(variant=TILED, N=33), dict(T=1 << 30, n=1), dict(C=(1 << 23) + 2), dict(n=1 << 30, T=0),
])
def test_scan_past_a_grid_is_unsupported(lib, change):  # noqa: F811
    call = {**SCAN, **EQUAL, **change}
    assert lib.conv_selective_scan_fwd(*call.values()) == cf.CONV_ERR_UNSUPPORTED
    assert cf.selective_scan_workspace(*(call[k] for k in ("T", "n", "C", "G", "N")), variant=call["variant"]) == -1


@pytest.mark.parametrize("change", [
    dict(variant=DIRECT, T=1 << 22, n=1 << 22, H=4, P=32),      # a wave takes 8 rows
    dict(variant=AUTO, T=1 << 22, n=1 << 22, H=4, P=32),
    dict(variant=TILED, T=1 << 22, n=1 << 22, H=64, G=4, P=64, ds=64),
    dict(variant=TILED, N=129, dt=cf.CONV_F32), dict(T=1 << 30, n=1), dict(H=65536), dict(P=65537),
])
def test_heads_past_a_grid_are_unsupported(lib, change):  # noqa: F811
    call = {**HEADS, **EQUAL, **change}
    assert lib.conv_selective_scan_heads_fwd(*call.values()) == cf.CONV_ERR_UNSUPPORTED
    sizes = (call[k] for k in ("T", "n", "H", "P", "G", "N", "dt", "variant"))
    assert lib.conv_selective_scan_heads_workspace(*sizes) == -1


@pytest.mark.parametrize("call,fn", [(SCAN, "conv_selective_scan"), (HEADS, "conv_selective_scan_heads")])
def test_workspace_too_small(lib, call, fn):  # noqa: F811
    """The workspace that the query asks for, and no byte less."""
    call = {**call, **EQUAL, "T": 3000, "n": 1, "variant": TILED}
    names = ("T", "n", "C", "G", "N", "dt", "variant") if "C" in call else ("T", "n", "H", "P", "G", "N", "dt", "variant")
    need = getattr(lib, fn + "_workspace")(*(call[k] for k in names))
    assert need > 0
    assert getattr(lib, fn + "_fwd")(*{**call, "wsb": need - 1}.values()) == cf.CONV_ERR_SHAPE
    assert getattr(lib, fn + "_fwd")(*{**call, "ws": None, "wsb": 0}.values()) == cf.CONV_ERR_NULL
    # No workspace for sequences of one segment, nor token by token.
    assert getattr(lib, fn + "_workspace")(*(dict(call, T=200)[k] for k in names)) == 0
    assert getattr(lib, fn + "_workspace")(*(dict(call, variant=DIRECT)[k] for k in names)) == 0


def test_rules_for_short_sequences(lib):  # noqa: F811
    """Where nothing is asked for, short sequences go token by token: no workspace, and states tiles do not take."""
    assert cf.selective_scan_workspace(3000, 1, 64, 1, 16) > 0
    assert cf.selective_scan_workspace(3000, 1000, 64, 1, 16) == 0
    assert cf.selective_scan_workspace(3000, 1, 64, 1, 64) == 0
    assert cf.selective_scan_heads_workspace(3000, 1, 4, 64, 1, 128) > 0
    assert cf.selective_scan_heads_workspace(3000, 1000, 4, 64, 1, 128) == 0
