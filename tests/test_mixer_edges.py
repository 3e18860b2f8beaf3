"""The token-mixer operators on the host: what the compiled code assumes, and the limits of what a call accepts."""
import importlib.util
import re
import subprocess
import sys

import pytest

import convolution_forward_amd as cf
from convolution_forward_amd import build
from test_mixer_abi import CONV, DELTA, PRODUCT, lib  # noqa: F401  (fake addresses: nothing may be launched)


def test_conv_promises_no_more_alignment_than_is_checked(tmp_path):
    """The four-channel bf16 form is chosen for 8-byte alignment: no global load or store of it may assume more."""
    out = tmp_path / "conv.ll"
    subprocess.run([build.HIPCC, *build.COMMON_FLAGS, "--offload-device-only", "-S", "-emit-llvm",
                    build.CSRC + "/causal_conv1d.hip", "-o", str(out)], check=True, capture_output=True)
    seen = 0
    for body in re.findall(r"^define .*?^}", out.read_text(), re.S | re.M):
        form = re.search(r"causal_conv1d_kernelI(\w)Li(\d)ELi\dE", body)
        if not form:
            continue
        most = int(form[2]) * {"t": 2, "f": 4}[form[1]]
        aligned = [int(a) for a in re.findall(r"(?:load|store) .*?addrspace\(1\).*?align (\d+)", body)]
        assert aligned and max(aligned) <= max(most, 4), form[0]    # (biases and offsets are 4-byte values)
        seen += 1
    assert seen == 28       # two types, two widths, 2 to 8 taps


@pytest.mark.parametrize("variant", [cf.VARIANT_AUTO, cf.VARIANT_DIRECT])
def test_delta_past_a_grid_is_unsupported(lib, variant):  # noqa: F811
    """Token by token a wave takes 32 columns of single tokens and 16 of others: 2^26 waves are 2^32 threads."""
    n = 1 << 20
    sizes = dict(T=n, n=n, Hk=2, Hv=4, Dk=64, Dv=512)
    call = {**DELTA, **sizes, "off": None, "slots": None, "si": None, "so": None, "variant": variant}
    assert lib.conv_delta_rule_fwd(*call.values()) == cf.CONV_ERR_UNSUPPORTED
    assert cf.delta_rule_workspace(*sizes.values(), variant=variant) == -1
    assert cf.delta_rule_workspace(n, n, 2, 4, 64, 480, variant=variant) == 0
    assert cf.delta_rule_workspace(8 * n, n, 2, 4, 64, 256, variant=variant) == -1
    assert cf.delta_rule_workspace(8 * n, n, 2, 4, 64, 240, variant=variant) == 0


@pytest.mark.parametrize("change", [dict(T=1 << 29, C=16, xs=16, ys=16), dict(C=(1 << 23) + 8, xs=1 << 24, ys=1 << 24)])
def test_conv_past_a_grid_is_unsupported(lib, change):  # noqa: F811
    call = {**CONV, "si": None, "so": None, **change}
    assert lib.conv_causal1d_fwd(*call.values()) == cf.CONV_ERR_UNSUPPORTED


@pytest.mark.parametrize("change", [dict(M=1 << 23, N=1 << 17, ys=1 << 17), dict(xs=(1 << 22) + 1), dict(ws=(1 << 22) + 1)])
def test_product_tiles_past_their_limits_are_unsupported(lib, change):  # noqa: F811
    call = {**PRODUCT, "b": None, **change, "variant": cf.VARIANT_TILED}
    assert lib.conv_matmul_q8_fwd(*call.values()) == cf.CONV_ERR_UNSUPPORTED


def test_import_leaves_torch_alone():
    """The C library's handle and constants need no torch; the mixer's names are there all the same."""
    code = ("import sys, convolution_forward_amd as cf; assert 'torch' not in sys.modules; cf.load_library; "
            "assert 'matmul_q8' in dir(cf) and not hasattr(cf, 'matmul_q9') and 'torch' not in sys.modules; "
            "from convolution_forward_amd import rms_norm_q8; assert cf.rms_norm_q8 is rms_norm_q8 is cf.mixer.rms_norm_q8")
    r = subprocess.run([sys.executable, "-c", code], cwd=build.ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_build_without_torch(monkeypatch, tmp_path):
    """Without torch there is no binding to build, and the C library's build goes on."""
    monkeypatch.setattr(build, "_compile", lambda src, incremental: src)
    linked = []

    def run(cmd, **kw):
        open(cmd[cmd.index("-o") + 1], "w").close()
        linked.append(cmd)
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setitem(sys.modules, "torch", None)
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: None)
    monkeypatch.setattr(build, "LIB_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libconvfwd.so"))
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "_mixer.so"))
    build.build()
    assert len(linked) == 1


def test_incremental_build_notices_another_torch(monkeypatch, tmp_path):
    import torch
    made = []

    def run(cmd, **kw):
        open(cmd[cmd.index("-o") + 1], "w").close()
        made.append(cmd)
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "_mixer.so"))
    monkeypatch.setattr(build, "BINDING_STAMP", str(tmp_path / "stamp"), raising=False)
    for version, builds in (("1", 1), ("1", 1), ("2", 2)):
        monkeypatch.setattr(torch, "__version__", version)
        build.build_binding(incremental=True)
        assert len(made) == builds
