"""Token-mixer operators: RMS norm with 8-bit output, 8-bit matrix product,
causal convolution and gated delta rule over packed sequences.

Argument marshalling only, like the rest of the package; include/convfwd.h
holds the definitions. Rows are tokens. The sequence operators take either
[batch, length, ...] tensors (equal lengths), or [tokens, ...] tensors with
``seq_offsets``, an int32 tensor on the GPU whose entries n and n+1 bound
sequence n's rows ([tokens, ...] without it is one sequence).
"""
from __future__ import annotations

import ctypes

import torch

from . import (CONV_BF16, CONV_E4M3, CONV_F32, CONV_I8, VARIANT_AUTO, _check, _stream_of, load_library)

_Strides = ctypes.c_int64 * 2

_FLOAT = {torch.float32: CONV_F32, torch.bfloat16: CONV_BF16}
_EIGHT = {torch.int8: CONV_I8, torch.float8_e4m3fn: CONV_E4M3}


def _code(table, t, what):
    code = table.get(t)
    if code is None:
        raise ValueError(f"{what}: unsupported dtype {t}; use {' or '.join(str(k) for k in table)}")
    return code


def _same_gpu(first, *others):
    """The GPU's index, the same for every tensor."""
    gpu = first.get_device()
    if gpu < 0:
        raise ValueError("tensors must live on the GPU (no CPU path exists)")
    for t in others:
        if t is not None and t.get_device() != gpu:
            raise ValueError(f"tensors on {first.device} and {t.device}: all must be on one GPU")
    return gpu


def _empty(like, shape, dtype):
    """A new contiguous tensor on `like`'s GPU."""
    if like.is_contiguous():
        return torch.empty_like(like, dtype=dtype)
    return like.new_empty(shape, dtype=dtype)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _vector(t, n, dtype, what):
    if t is not None and (t.dtype != dtype or t.numel() != n or not t.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of {n} values")


def _rows(t, what, width=None, rows=None, dtype=None):
    """Row stride of a [rows, width] tensor whose channels are adjacent."""
    shape = t.shape
    if len(shape) == 2 and (width is None or shape[1] == width) and (rows is None or shape[0] == rows) and \
            (dtype is None or t.dtype == dtype):
        if t.is_contiguous():
            return shape[1]
        if t.stride(1) == 1 or shape[1] == 1:
            return t.stride(0) if shape[0] > 1 else max(t.stride(0), shape[1])
    raise ValueError(f"{what} must be [{'rows' if rows is None else rows}, {'width' if width is None else width}]"
                     f"{'' if dtype is None else f' {dtype}'} with adjacent channels, got {tuple(shape)} {t.dtype}"
                     f" with strides {t.stride()}")


def _flat(t):
    """[..., channels] as [rows, channels] without a copy."""
    if t.dim() == 2:
        return t
    try:
        return t.view(-1, t.shape[-1])
    except RuntimeError as e:
        raise ValueError(f"rows of shape {tuple(t.shape)}, strides {t.stride()} are not evenly spaced") from e


def rms_norm_q8(x, weight, residual=None, eps: float = 1e-6, out_dtype=torch.int8, out=None, scale=None, sum_out=None):
    """RMS norm of x (+ residual), quantised to 8 bits with one scale a row.

    x, residual [..., width] float32 or bfloat16; weight [width] of the same
    type; out_dtype torch.int8 or torch.float8_e4m3fn. Returns (q, scale, h):
    q like x in 8 bits, scale [...] float32 with q * scale the normed values,
    h = x + residual (None without a residual). sum_out may be x or residual.
    """
    lib = load_library()
    gpu = _same_gpu(x, weight, residual, out, scale, sum_out)
    dt = _code(_FLOAT, x.dtype, "x")
    width = x.shape[-1]
    x2 = _flat(x)
    rows = x2.shape[0]
    xs = _rows(x2, "x")
    _vector(weight, width, x.dtype, "weight")
    rs = hs = 0
    r2 = h2 = None
    if residual is not None:
        r2 = _flat(residual)
        rs = _rows(r2, "residual", width, rows, x.dtype)
        if sum_out is None:
            sum_out = _empty(x, x.shape, x.dtype)
        h2 = _flat(sum_out)
        hs = _rows(h2, "sum_out", width, rows, x.dtype)
    elif sum_out is not None:
        raise ValueError("sum_out without a residual")
    if out is None:
        out = _empty(x, x.shape, out_dtype)
    q2 = _flat(out)
    qs = _rows(q2, "out", width, rows)
    qdt = _code(_EIGHT, out.dtype, "out")
    if scale is None:
        scale = x.new_empty(x.shape[:-1], dtype=torch.float32)
    else:
        _vector(scale, rows, torch.float32, "scale")
    _check(lib.conv_rms_norm_q8_fwd(x2.data_ptr(), xs, _ptr(r2), rs, weight.data_ptr(), _ptr(h2), hs, q2.data_ptr(), qs,
                                    scale.data_ptr(), rows, width, eps, dt, qdt, _stream_of(gpu)),
           "conv_rms_norm_q8_fwd")
    return out, scale, sum_out


def matmul_q8(x, x_scale, w, w_scale, bias=None, out_dtype=torch.bfloat16, out=None, variant: int = VARIANT_AUTO):
    """y[..., n] = x_scale * w_scale[n] * (x . w[n]) + bias[n] for 8-bit x and w.

    x [..., K] and w [N, K] torch.int8 or torch.float8_e4m3fn (the same),
    x_scale [...] and w_scale [N] float32, bias [N] float32; out_dtype
    torch.bfloat16 or torch.float32.
    """
    lib = load_library()
    gpu = _same_gpu(x, x_scale, w, w_scale, bias, out)
    q = _code(_EIGHT, x.dtype, "x")
    x2 = _flat(x)
    M, K = x2.shape
    xs = _rows(x2, "x")
    ws = _rows(w, "w", K, None, x.dtype)
    N = w.shape[0]
    _vector(x_scale, M, torch.float32, "x_scale")
    _vector(w_scale, N, torch.float32, "w_scale")
    _vector(bias, N, torch.float32, "bias")
    if out is None:
        out = x.new_empty(x.shape[:-1] + (N,), dtype=out_dtype)
    y2 = _flat(out)
    ys = _rows(y2, "out", N, M)
    _check(lib.conv_matmul_q8_fwd(x2.data_ptr(), xs, x_scale.data_ptr(), w.data_ptr(), ws, w_scale.data_ptr(), _ptr(bias),
                                  y2.data_ptr(), ys, M, N, K, q, _code(_FLOAT, out.dtype, "out"), variant,
                                  _stream_of(gpu)), "conv_matmul_q8_fwd")
    return out


def _sequences(t, tail, seq_offsets):
    """(tokens, sequences) of a tensor [batch, length, ...] or [tokens, ...]
    whose last `tail` axes are not tokens."""
    if t.dim() == tail + 2:
        if seq_offsets is not None:
            raise ValueError("seq_offsets go with [tokens, ...] tensors")
        return t.shape[0] * t.shape[1], t.shape[0]
    if t.dim() != tail + 1:
        raise ValueError(f"expected [batch, length, ...] or [tokens, ...], got {tuple(t.shape)}")
    if seq_offsets is None:
        return t.shape[0], 1
    if seq_offsets.dtype != torch.int32 or seq_offsets.dim() != 1 or seq_offsets.numel() < 2 or \
            not seq_offsets.is_contiguous():
        raise ValueError("seq_offsets must be a contiguous int32 tensor of num_seqs + 1 values")
    return t.shape[0], seq_offsets.numel() - 1


def _states(initial, final, shape, dtype, slots, num_seqs):
    """Slots of the state tensors, [num_slots, *shape]."""
    num = 0
    for t in (initial, final):
        if t is None:
            continue
        if t.dtype != dtype or tuple(t.shape[1:]) != shape or not t.is_contiguous():
            raise ValueError(f"states must be contiguous {dtype} tensors [slots, {', '.join(map(str, shape))}]")
        if num and t.shape[0] != num:
            raise ValueError("initial_state and final_state must have as many slots")
        num = t.shape[0]
    _vector(slots, num_seqs, torch.int32, "slots")
    return num


def causal_conv1d(x, w, bias=None, activation=None, seq_offsets=None, initial_state=None, final_state=None, slots=None,
                  out=None):
    """Causal depthwise convolution along each sequence, with carried state.

    x [batch, length, channels] or [tokens, channels]; w [channels, taps] of
    x's type (2 to 8 taps, the last one the token's own); bias [channels]
    float32; activation None or "silu". initial_state and final_state
    [slots, taps-1, channels] of x's type, possibly the same tensor.
    """
    lib = load_library()
    gpu = _same_gpu(x, w, bias, seq_offsets, initial_state, final_state, slots, out)
    dt = _code(_FLOAT, x.dtype, "x")
    if activation not in (None, "silu"):
        raise ValueError(f"activation {activation!r}: None or 'silu'")
    tokens, seqs = _sequences(x, 1, seq_offsets)
    C = x.shape[-1]
    if w.dim() != 2 or w.shape[0] != C or w.dtype != x.dtype or not w.is_contiguous():
        raise ValueError(f"w must be a contiguous [{C}, taps] tensor of {x.dtype}")
    taps = w.shape[1]
    _vector(bias, C, torch.float32, "bias")
    num = _states(initial_state, final_state, (taps - 1, C), x.dtype, slots, seqs)
    x2 = _flat(x)
    if out is None:
        out = _empty(x, x.shape, x.dtype)
    y2 = _flat(out)
    ys = _rows(y2, "out", C, tokens, x.dtype)
    _check(lib.conv_causal1d_fwd(x2.data_ptr(), _rows(x2, "x"), w.data_ptr(), _ptr(bias), y2.data_ptr(), ys,
                                 _ptr(seq_offsets), _ptr(initial_state), _ptr(final_state), _ptr(slots), num, tokens,
                                 seqs, C, taps, activation == "silu", dt, _stream_of(gpu)), "conv_causal1d_fwd")
    return out


def _heads(t, tokens, what, heads=None, width=None, dtype=None):
    """(token, head) strides of [tokens, heads, width], tokens possibly over two axes."""
    if t.dim() == 4:
        b, n = t.shape[:2]
        if b > 1 and n > 1 and t.stride(0) != n * t.stride(1):
            raise ValueError(f"{what}: batch and length of strides {t.stride()} are not one row of tokens")
        st = t.stride(1) if n > 1 else t.stride(0)
    else:
        st = t.stride(0)
    if (heads is not None and t.shape[-2] != heads) or (width is not None and t.shape[-1] != width) or \
            (t.stride(-1) != 1 and t.shape[-1] > 1) or (dtype is not None and t.dtype != dtype) or \
            t.numel() != tokens * t.shape[-2] * t.shape[-1]:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, strides {t.stride()}, {t.dtype} do not fit the other tensors")
    return _Strides(st, t.stride(-2))


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
    """
    lib = load_library()
    gpu = _same_gpu(q, k, v, g, beta, seq_offsets, initial_state, final_state, slots, out, workspace)
    dt = _code(_FLOAT, q.dtype, "q")
    tokens, seqs = _sequences(q, 2, seq_offsets)
    Hk, Dk = q.shape[-2:]
    Hv, Dv = v.shape[-2:]
    sq = _heads(q, tokens, "q")
    sk = _heads(k, tokens, "k", Hk, Dk, q.dtype)
    sv = _heads(v, tokens, "v", Hv, Dv, q.dtype)
    _vector(g, tokens * Hv, torch.float32, "g")
    _vector(beta, tokens * Hv, torch.float32, "beta")
    num = _states(initial_state, final_state, (Hv, Dk, Dv), torch.float32, slots, seqs)
    if out is None:
        out = _empty(v, v.shape, v.dtype)
    so = _heads(out, tokens, "out", Hv, Dv, q.dtype)
    if workspace is None:
        need = lib.conv_delta_rule_workspace(tokens, seqs, Hk, Hv, Dk, Dv, dt, variant)
        if need > 0:
            workspace = q.new_empty(need, dtype=torch.uint8)
    _check(lib.conv_delta_rule_fwd(q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, g.data_ptr(), beta.data_ptr(),
                                   _ptr(seq_offsets), _ptr(initial_state), _ptr(final_state), _ptr(slots), num,
                                   out.data_ptr(), so, _ptr(workspace),
                                   0 if workspace is None else workspace.numel() * workspace.element_size(), tokens, seqs,
                                   Hk, Hv, Dk, Dv, Dk ** -0.5 if scale is None else scale, bool(normalize), dt, variant,
                                   _stream_of(gpu)), "conv_delta_rule_fwd")
    return out


def delta_rule_workspace(tokens: int, num_seqs: int, Hk: int, Hv: int, Dk: int, Dv: int, dtype=torch.bfloat16,
                         variant: int = VARIANT_AUTO) -> int:
    """Bytes of workspace gated_delta_rule needs for these sizes."""
    return int(load_library().conv_delta_rule_workspace(tokens, num_seqs, Hk, Hv, Dk, Dv,
                                                        _code(_FLOAT, dtype, "dtype"), variant))
