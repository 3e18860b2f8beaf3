"""Token-mixer operators: RMS norm with 8-bit output, 8-bit matrix product,
causal convolution and gated delta rule over packed sequences.

include/convfwd.h holds the definitions; the arguments are marshalled by a
small compiled binding (binding/mixer_binding.cpp), since a single token's
kernel takes less time than the same checks in Python. Rows are tokens. The
sequence operators take either [batch, length, ...] tensors (equal lengths),
or [tokens, ...] tensors with ``seq_offsets``, an int32 tensor on the GPU whose
entries n and n+1 bound sequence n's rows ([tokens, ...] without it is one
sequence).
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os

import torch

from . import _PKG, CONV_BF16, CONV_F32, VARIANT_AUTO, _check, load_library

BINDING_PATH = os.path.join(_PKG, "_lib", "_mixer.so")
_binding = None


def _load():
    global _binding
    load_library()      # says how to build where nothing is built
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"{BINDING_PATH} is not built; run `python -m convolution_forward_amd.build`")
    loader = importlib.machinery.ExtensionFileLoader("_mixer", BINDING_PATH)
    _binding = importlib.util.module_from_spec(importlib.util.spec_from_loader("_mixer", loader))
    loader.exec_module(_binding)
    return _binding


def rms_norm_q8(x, weight, residual=None, eps: float = 1e-6, out_dtype=torch.int8, out=None, scale=None, sum_out=None):
    """RMS norm of x (+ residual), quantised to 8 bits with one scale a row.

    x, residual [..., width] float32 or bfloat16; weight [width] of the same
    type; out_dtype torch.int8 or torch.float8_e4m3fn. Returns (q, scale, h):
    q like x in 8 bits, scale [...] float32 with q * scale the normed values,
    h = x + residual (None without a residual). sum_out may be x or residual.
    """
    r = (_binding or _load()).rms_norm_q8(x, weight, residual, eps, out_dtype, out, scale, sum_out)
    if type(r) is int:
        _check(r, "conv_rms_norm_q8_fwd")
    return r


def matmul_q8(x, x_scale, w, w_scale, bias=None, out_dtype=torch.bfloat16, out=None, variant: int = VARIANT_AUTO):
    """y[..., n] = x_scale * w_scale[n] * (x . w[n]) + bias[n] for 8-bit x and w.

    x [..., K] and w [N, K] torch.int8 or torch.float8_e4m3fn (the same),
    x_scale [...] and w_scale [N] float32, bias [N] float32; out_dtype
    torch.bfloat16 or torch.float32.
    """
    r = (_binding or _load()).matmul_q8(x, x_scale, w, w_scale, bias, out_dtype, out, variant)
    if type(r) is int:
        _check(r, "conv_matmul_q8_fwd")
    return r


def causal_conv1d(x, w, bias=None, activation=None, seq_offsets=None, initial_state=None, final_state=None, slots=None,
                  out=None):
    """Causal depthwise convolution along each sequence, with carried state.

    x [batch, length, channels] or [tokens, channels]; w [channels, taps] of
    x's type (2 to 8 taps, the last one the token's own); bias [channels]
    float32; activation None or "silu". initial_state and final_state
    [slots, taps-1, channels] of x's type, possibly the same tensor.
    """
    if activation is not None and activation != "silu":
        raise ValueError(f"activation {activation!r}: None or 'silu'")
    r = (_binding or _load()).causal_conv1d(x, w, bias, activation is not None, seq_offsets, initial_state, final_state,
                                            slots, out)
    if type(r) is int:
        _check(r, "conv_causal1d_fwd")
    return r


def gated_delta_rule(q, k, v, g, beta, scale=None, normalize: bool = False, seq_offsets=None, initial_state=None,
                     final_state=None, slots=None, out=None, workspace=None, variant: int = VARIANT_AUTO):
    """The gated delta rule along each sequence (conv_delta_rule_fwd in include/convfwd.h).

    q, k [batch, length, Hk, Dk] or [tokens, Hk, Dk]; v [..., Hv, Dv] of the
    same type (float32 or bfloat16), Hv a multiple of Hk; g (log decay) and
    beta [..., Hv] float32. scale defaults to Dk ** -0.5; normalize divides q
    and k by their 2-norms first. initial_state and final_state
    [slots, Hv, Dk, Dv] float32, possibly the same tensor. workspace: a uint8
    tensor of at least delta_rule_workspace(...) bytes; without it one is
    taken from torch's allocator for the call. Returns o like v.

    VARIANT_AUTO chooses between chunks and single steps for the whole call,
    by its mean length: a prompt is best kept apart from many single tokens.
    """
    r = (_binding or _load()).gated_delta_rule(q, k, v, g, beta, scale, normalize, seq_offsets, initial_state, final_state,
                                               slots, out, workspace, variant)
    if type(r) is int:
        _check(r, "conv_delta_rule_fwd")
    return r


def delta_rule_workspace(tokens: int, num_seqs: int, Hk: int, Hv: int, Dk: int, Dv: int, dtype=torch.bfloat16,
                         variant: int = VARIANT_AUTO) -> int:
    """Bytes of workspace gated_delta_rule needs for these sizes (-1: the sizes are an error)."""
    code = {torch.float32: CONV_F32, torch.bfloat16: CONV_BF16}.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}; use float32 or bfloat16")
    return int(load_library().conv_delta_rule_workspace(tokens, num_seqs, Hk, Hv, Dk, Dv, code, variant))
