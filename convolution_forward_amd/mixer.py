"""Token-mixer operators: RMS norm with 8-bit output, 8-bit matrix product,
causal convolution, head norms with rotation, gated delta rule and selective
scans over packed sequences.

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
import math
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


def rotary(q, positions, frequencies, k=None, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
           scale: float = 1.0, out=None, k_out=None):
    """Norms of queries and keys for each head, and their rotation by position (conv_rotary_fwd in include/convfwd.h).

    q [tokens, Hq, D] or [batch, length, Hq, D] float32 or bfloat16, k likewise
    with Hk heads; positions [tokens] or [batch, length], contiguous, int64 or
    int32; frequencies [R / 2] float32, as rotary_frequencies
    makes them: the first R values of a head are rotated, in pairs i and
    i + R/2, or 2i and 2i + 1 with interleaved. q_weight and k_weight [D] of
    q's type: an RMS norm before the rotation; without one the values are
    rotated as they are. scale multiplies what is rotated. out and k_out may be
    q and k. Returns q's result, with k a pair.
    """
    r = (_binding or _load()).rotary(q, positions, frequencies, k, q_weight, k_weight, eps, interleaved, scale, out, k_out)
    if type(r) is int:
        _check(r, "conv_rotary_fwd")
    return r


def rotary_frequencies(rotated: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       trained: int = 0, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """(frequencies [rotated / 2] float32, scale) for rotary: base ** (-2 i / rotated), stretched for long contexts.

    scaling None: as they are. "linear": divided by factor. "base": the base
    raised so that the slowest frequency is divided by factor and the fastest
    is kept. "parts": frequencies of at most `slow` turns in `trained`
    positions divided by factor, those of at least `fast` turns kept, and a ramp
    over the turns' logarithm (over the index i) between; the scale is then
    0.1 ln(factor) + 1. "wavelength": the same bounds, a ramp over the turns
    themselves, and scale 1. Computed in 64 bits on the host.
    """
    if rotated <= 0 or rotated % 2:
        raise ValueError(f"rotated {rotated}: a positive even number")
    if scaling not in (None, "linear", "base", "parts", "wavelength"):
        raise ValueError(f"scaling {scaling!r}: None, 'linear', 'base', 'parts' or 'wavelength'")
    if not (base > 1.0 and factor >= 1.0):
        raise ValueError(f"base {base} must be above 1 and factor {factor} at least 1")
    if scaling in ("parts", "wavelength") and not (trained > 0 and fast > slow > 0.0):
        raise ValueError(f"{scaling} needs trained > 0 and fast > slow > 0, got {trained}, {fast} and {slow}")
    half = rotated // 2
    if scaling == "base" and half > 1:
        base *= factor ** (half / (half - 1))
    f = [base ** (-i / half) for i in range(half)]
    scale = 1.0
    if scaling == "linear" or (scaling == "base" and half == 1):
        f = [v / factor for v in f]
    elif scaling in ("parts", "wavelength"):
        if scaling == "parts":
            # The index at which a frequency makes that many turns.
            ends = [half * math.log(trained / (2 * math.pi * turns)) / math.log(base) for turns in (fast, slow)]
            lo, hi = max(math.floor(ends[0]), 0), min(math.ceil(ends[1]), rotated - 1)
            # hi is past lo unless one was moved into the range: then all make at most `slow` turns, or `fast` and more.
            keep = [1.0 - min(max((i - lo) / (hi - lo), 0.0), 1.0) if hi > lo else float(i < lo) for i in range(half)]
            scale = 0.1 * math.log(factor) + 1.0
        else:
            keep = [min(max((trained * v / (2 * math.pi) - slow) / (fast - slow), 0.0), 1.0) for v in f]
        f = [v * (k + (1.0 - k) / factor) for v, k in zip(f, keep)]
    return torch.tensor(f, dtype=torch.float64).float().to(device), scale


def selective_scan(x, dt, a, b, c, skip=None, gate=None, dt_bias=None, dt_softplus: bool = False, seq_offsets=None,
                   initial_state=None, final_state=None, slots=None, out=None, workspace=None, variant: int = VARIANT_AUTO):
    """The selective state space scan with a decay for each channel and state (conv_selective_scan_fwd in
    include/convfwd.h).

    x, dt, gate [batch, length, channels] or [tokens, channels] float32 or
    bfloat16; a [channels, states] float32; b, c [..., groups, states] of x's
    type, channels a multiple of groups; skip, dt_bias [channels] float32.
    initial_state and final_state [slots, channels, states] float32, possibly
    the same tensor. workspace: a uint8 tensor of at least
    selective_scan_workspace(...) bytes; without it one is taken from torch's
    allocator for the call. Returns y like x.

    VARIANT_AUTO chooses between tiles (up to 32 states) and single steps for
    the whole call, by its mean length: a prompt is best kept apart from many
    single tokens.
    """
    r = (_binding or _load()).selective_scan(x, dt, a, b, c, skip, gate, dt_bias, dt_softplus, seq_offsets, initial_state,
                                             final_state, slots, out, workspace, variant)
    if type(r) is int:
        _check(r, "conv_selective_scan_fwd")
    return r


def selective_scan_heads(x, dt, a, b, c, skip=None, gate=None, dt_bias=None, dt_softplus: bool = False, seq_offsets=None,
                         initial_state=None, final_state=None, slots=None, out=None, workspace=None,
                         variant: int = VARIANT_AUTO):
    """The selective state space scan with one decay a head (conv_selective_scan_heads_fwd in include/convfwd.h).

    x, gate [batch, length, H, P] or [tokens, H, P] float32 or bfloat16;
    dt [..., H] and b, c [..., groups, states] of x's type, H a multiple of
    groups; a, skip, dt_bias [H] float32. initial_state and final_state
    [slots, H, P, states] float32, possibly the same tensor. workspace: a uint8
    tensor of at least selective_scan_heads_workspace(...) bytes; without it one
    is taken from torch's allocator for the call. Returns y like x.

    VARIANT_AUTO chooses between chunks (float32: up to 128 states) and single
    steps for the whole call, by its mean length, as in selective_scan.
    """
    r = (_binding or _load()).selective_scan_heads(x, dt, a, b, c, skip, gate, dt_bias, dt_softplus, seq_offsets,
                                                   initial_state, final_state, slots, out, workspace, variant)
    if type(r) is int:
        _check(r, "conv_selective_scan_heads_fwd")
    return r


def _float_code(dtype) -> int:
    code = {torch.float32: CONV_F32, torch.bfloat16: CONV_BF16}.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}; use float32 or bfloat16")
    return code


def selective_scan_workspace(tokens: int, num_seqs: int, channels: int, groups: int, states: int, dtype=torch.bfloat16,
                             variant: int = VARIANT_AUTO) -> int:
    """Bytes of workspace selective_scan needs for these sizes (-1: the sizes are an error)."""
    return int(load_library().conv_selective_scan_workspace(tokens, num_seqs, channels, groups, states, _float_code(dtype),
                                                            variant))


def selective_scan_heads_workspace(tokens: int, num_seqs: int, H: int, P: int, groups: int, states: int,
                                   dtype=torch.bfloat16, variant: int = VARIANT_AUTO) -> int:
    """Bytes of workspace selective_scan_heads needs for these sizes (-1: the sizes are an error)."""
    return int(load_library().conv_selective_scan_heads_workspace(tokens, num_seqs, H, P, groups, states,
                                                                  _float_code(dtype), variant))
