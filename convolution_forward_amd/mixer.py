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


# A call's host time counts where the kernel takes a few microseconds (single tokens), so the checks below ask each
# tensor as little as they can: one shape, one stride tuple, one data pointer.


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
    """A new contiguous tensor on `like`'s GPU (empty_like is the cheaper call where it gives just that)."""
    if like.shape == shape and like.is_contiguous():
        return torch.empty_like(like, dtype=dtype)
    return torch.empty(shape, dtype=dtype, device=like.device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _vector(t, n, dtype, what):
    """Data pointer of a contiguous vector of n values, or None."""
    if t is None:
        return None
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of {n} values")
    return t.data_ptr()


def _rows(t, what, width, rows=None, dtype=None):
    """(rows, row stride) of a [..., width] tensor whose channels are adjacent and whose rows are evenly spaced."""
    shape = t.shape
    if shape[-1] == width and (dtype is None or t.dtype == dtype):
        n = 1
        for size in shape[:-1]:
            n *= size
        if rows is None or n == rows:
            if t.is_contiguous():
                return n, width
            strides = t.stride()
            if strides[-1] == 1 or width == 1:
                step = 0        # from the innermost axis of more than one row outwards, each must continue the last
                for size, stride in zip(shape[-2::-1], strides[-2::-1]):
                    if size == 1:
                        continue
                    if step and stride != step * count:
                        break
                    step, count = (step or stride), (count * size if step else size)
                else:
                    return n, max(step, width) if n <= 1 else step
    raise ValueError(f"{what} must be [{'rows' if rows is None else rows}, {width}]{'' if dtype is None else f' {dtype}'}"
                     f" with adjacent channels and evenly spaced rows, got {tuple(shape)} {t.dtype}"
                     f" with strides {t.stride()}")


def rms_norm_q8(x, weight, residual=None, eps: float = 1e-6, out_dtype=torch.int8, out=None, scale=None, sum_out=None):
    """RMS norm of x (+ residual), quantised to 8 bits with one scale a row.

    x, residual [..., width] float32 or bfloat16; weight [width] of the same
    type; out_dtype torch.int8 or torch.float8_e4m3fn. Returns (q, scale, h):
    q like x in 8 bits, scale [...] float32 with q * scale the normed values,
    h = x + residual (None without a residual). sum_out may be x or residual.
    """
    gpu = _same_gpu(x, weight, residual, out, scale, sum_out)
    dtype, shape = x.dtype, x.shape
    dt = _code(_FLOAT, dtype, "x")
    width = shape[-1]
    rows, xs = _rows(x, "x", width)
    wp = _vector(weight, width, dtype, "weight")
    rp = hp = None
    rs = hs = 0
    if residual is not None:
        _, rs = _rows(residual, "residual", width, rows, dtype)
        rp = residual.data_ptr()
        if sum_out is None:
            sum_out, hs = _empty(x, shape, dtype), width
        else:
            _, hs = _rows(sum_out, "sum_out", width, rows, dtype)
        hp = sum_out.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out without a residual")
    if out is None:
        qdt = _code(_EIGHT, out_dtype, "out_dtype")
        out, qs = _empty(x, shape, out_dtype), width
    else:
        qdt = _code(_EIGHT, out.dtype, "out")
        _, qs = _rows(out, "out", width, rows)
    if scale is None:
        scale = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
        sp = scale.data_ptr()
    else:
        sp = _vector(scale, rows, torch.float32, "scale")
    st = load_library().conv_rms_norm_q8_fwd(x.data_ptr(), xs, rp, rs, wp, hp, hs, out.data_ptr(), qs, sp, rows, width,
                                             eps, dt, qdt, _stream_of(gpu))
    if st:
        _check(st, "conv_rms_norm_q8_fwd")
    return out, scale, sum_out


def matmul_q8(x, x_scale, w, w_scale, bias=None, out_dtype=torch.bfloat16, out=None, variant: int = VARIANT_AUTO):
    """y[..., n] = x_scale * w_scale[n] * (x . w[n]) + bias[n] for 8-bit x and w.

    x [..., K] and w [N, K] torch.int8 or torch.float8_e4m3fn (the same),
    x_scale [...] and w_scale [N] float32, bias [N] float32; out_dtype
    torch.bfloat16 or torch.float32.
    """
    gpu = _same_gpu(x, x_scale, w, w_scale, bias, out)
    dtype, shape = x.dtype, x.shape
    q = _code(_EIGHT, dtype, "x")
    K = shape[-1]
    M, xs = _rows(x, "x", K)
    if w.dim() != 2:
        raise ValueError(f"w must be [channels, {K}], got {tuple(w.shape)}")
    N, ws = _rows(w, "w", K, None, dtype)
    sx = _vector(x_scale, M, torch.float32, "x_scale")
    sw = _vector(w_scale, N, torch.float32, "w_scale")
    bp = _vector(bias, N, torch.float32, "bias")
    if out is None:
        ydt = _code(_FLOAT, out_dtype, "out_dtype")
        out, ys = torch.empty(shape[:-1] + (N,), dtype=out_dtype, device=x.device), N
    else:
        ydt = _code(_FLOAT, out.dtype, "out")
        _, ys = _rows(out, "out", N, M)
    st = load_library().conv_matmul_q8_fwd(x.data_ptr(), xs, sx, w.data_ptr(), ws, sw, bp, out.data_ptr(), ys, M, N, K, q,
                                           ydt, variant, _stream_of(gpu))
    if st:
        _check(st, "conv_matmul_q8_fwd")
    return out


def _sequences(shape, tail, seq_offsets):
    """(tokens, sequences) of a tensor [batch, length, ...] or [tokens, ...]
    whose last `tail` axes are not tokens."""
    dim = len(shape) - tail
    if dim == 2:
        if seq_offsets is not None:
            raise ValueError("seq_offsets go with [tokens, ...] tensors")
        return shape[0] * shape[1], shape[0]
    if dim != 1:
        raise ValueError(f"expected [batch, length, ...] or [tokens, ...], got {tuple(shape)}")
    if seq_offsets is None:
        return shape[0], 1
    n = seq_offsets.numel()
    if seq_offsets.dtype != torch.int32 or n < 2 or seq_offsets.dim() != 1 or not seq_offsets.is_contiguous():
        raise ValueError("seq_offsets must be a contiguous int32 tensor of num_seqs + 1 values")
    return shape[0], n - 1


def _state(t, shape, dtype, num):
    """Slots of a state tensor [slots, *shape]; `num`, if any, is what another has."""
    if t is None:
        return num
    s = t.shape
    if t.dtype != dtype or s[1:] != shape or not t.is_contiguous():
        raise ValueError(f"states must be contiguous {dtype} tensors [slots, {', '.join(map(str, shape))}]")
    if num and s[0] != num:
        raise ValueError("initial_state and final_state must have as many slots")
    return s[0]


def causal_conv1d(x, w, bias=None, activation=None, seq_offsets=None, initial_state=None, final_state=None, slots=None,
                  out=None):
    """Causal depthwise convolution along each sequence, with carried state.

    x [batch, length, channels] or [tokens, channels]; w [channels, taps] of
    x's type (2 to 8 taps, the last one the token's own); bias [channels]
    float32; activation None or "silu". initial_state and final_state
    [slots, taps-1, channels] of x's type, possibly the same tensor.
    """
    gpu = _same_gpu(x, w, bias, seq_offsets, initial_state, final_state, slots, out)
    dtype, shape = x.dtype, x.shape
    dt = _code(_FLOAT, dtype, "x")
    if activation is not None and activation != "silu":
        raise ValueError(f"activation {activation!r}: None or 'silu'")
    tokens, seqs = _sequences(shape, 1, seq_offsets)
    C = shape[-1]
    ws = w.shape
    if len(ws) != 2 or ws[0] != C or w.dtype != dtype or not w.is_contiguous():
        raise ValueError(f"w must be a contiguous [{C}, taps] tensor of {dtype}")
    taps = ws[1]
    bp = _vector(bias, C, torch.float32, "bias")
    num = _state(initial_state, (taps - 1, C), dtype, 0)
    num = _state(final_state, (taps - 1, C), dtype, num)
    lp = _vector(slots, seqs, torch.int32, "slots")
    _, xs = _rows(x, "x", C)
    if out is None:
        out, ys = _empty(x, shape, dtype), C
    else:
        _, ys = _rows(out, "out", C, tokens, dtype)
    st = load_library().conv_causal1d_fwd(x.data_ptr(), xs, w.data_ptr(), bp, out.data_ptr(), ys, _ptr(seq_offsets),
                                          _ptr(initial_state), _ptr(final_state), lp, num, tokens, seqs, C, taps,
                                          activation is not None, dt, _stream_of(gpu))
    if st:
        _check(st, "conv_causal1d_fwd")
    return out


def _heads(t, tokens, what, heads, width, dtype):
    """(token, head) strides of [tokens, heads, width], tokens possibly over two axes."""
    shape, strides = t.shape, t.stride()
    if len(shape) == 4:
        b, n = shape[:2]
        if b > 1 and n > 1 and strides[0] != n * strides[1]:
            raise ValueError(f"{what}: batch and length of strides {strides} are not one row of tokens")
        rows, st = b * n, strides[1] if n > 1 else strides[0]
    else:
        rows, st = shape[0], strides[0]
    if len(shape) < 3 or rows != tokens or shape[-2] != heads or shape[-1] != width or t.dtype != dtype or \
            (strides[-1] != 1 and width > 1):
        raise ValueError(f"{what}: shape {tuple(shape)}, strides {strides}, {t.dtype} do not fit the other tensors")
    return _Strides(st, strides[-2])


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
    dtype, shape, vshape = q.dtype, q.shape, v.shape
    dt = _code(_FLOAT, dtype, "q")
    tokens, seqs = _sequences(shape, 2, seq_offsets)
    Hk, Dk = shape[-2], shape[-1]
    Hv, Dv = vshape[-2], vshape[-1]
    sq = _heads(q, tokens, "q", Hk, Dk, dtype)
    sk = _heads(k, tokens, "k", Hk, Dk, dtype)
    sv = _heads(v, tokens, "v", Hv, Dv, dtype)
    gp = _vector(g, tokens * Hv, torch.float32, "g")
    bp = _vector(beta, tokens * Hv, torch.float32, "beta")
    num = _state(initial_state, (Hv, Dk, Dv), torch.float32, 0)
    num = _state(final_state, (Hv, Dk, Dv), torch.float32, num)
    lp = _vector(slots, seqs, torch.int32, "slots")
    if out is None:
        out, so = torch.empty(vshape, dtype=dtype, device=v.device), None
    else:
        so = _heads(out, tokens, "out", Hv, Dv, dtype)
    wp, wbytes = None, 0
    if workspace is not None:
        wp, wbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    else:
        wbytes = lib.conv_delta_rule_workspace(tokens, seqs, Hk, Hv, Dk, Dv, dt, variant)
        if wbytes > 0:
            workspace = torch.empty(wbytes, dtype=torch.uint8, device=q.device)
            wp = workspace.data_ptr()
    st = lib.conv_delta_rule_fwd(q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, gp, bp, _ptr(seq_offsets),
                                 _ptr(initial_state), _ptr(final_state), lp, num, out.data_ptr(), so, wp, wbytes, tokens,
                                 seqs, Hk, Hv, Dk, Dv, Dk ** -0.5 if scale is None else scale, normalize, dt, variant,
                                 _stream_of(gpu))
    if st:
        _check(st, "conv_delta_rule_fwd")
    return out


def delta_rule_workspace(tokens: int, num_seqs: int, Hk: int, Hv: int, Dk: int, Dv: int, dtype=torch.bfloat16,
                         variant: int = VARIANT_AUTO) -> int:
    """Bytes of workspace gated_delta_rule needs for these sizes."""
    return int(load_library().conv_delta_rule_workspace(tokens, num_seqs, Hk, Hv, Dk, Dv,
                                                        _code(_FLOAT, dtype, "dtype"), variant))
