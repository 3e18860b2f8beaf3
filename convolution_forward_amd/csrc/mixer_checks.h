// Host-side argument checks that the token-mixer operators share.
#pragma once

#include <limits.h>
#include <stdint.h>

#include "checks.h"
#include "internal.h"

namespace convfwd {

inline bool is_float(conv_dtype d) { return d == CONV_F32 || d == CONV_BF16; }
inline bool is_eight(conv_dtype d) { return d == CONV_I8 || d == CONV_E4M3; }
inline int64_t size_of(conv_dtype d) { return d == CONV_F32 ? 4 : (d == CONV_BF16 ? 2 : 1); }
inline bool aligned(const void *p, int64_t to) { return (uintptr_t)p % (uintptr_t)to == 0; }

// Kernels index rows, tokens and tiles with int.
constexpr int64_t MAX_ROWS = INT_MAX / 2;

// Bytes of `rows` rows of `width` elements, `stride` apart, or -1 past
// MAX_EXTENT_BYTES. 0 rows touch nothing.
inline int64_t rows_bytes(int64_t rows, int64_t stride, int64_t width, int64_t esize)
{
    if (rows == 0)
        return 0;
    int64_t last, bytes;
    if (__builtin_mul_overflow(rows - 1, stride, &last) || __builtin_add_overflow(last, width, &last) ||
        __builtin_mul_overflow(last, esize, &bytes) || bytes > MAX_EXTENT_BYTES)
        return -1;
    return bytes;
}

// Bytes of a contiguous tensor of a*b*c*d elements, or -1.
inline int64_t flat_bytes(int64_t a, int64_t b, int64_t c, int64_t d, int64_t esize)
{
    int64_t n;
    if (__builtin_mul_overflow(a, b, &n) || __builtin_mul_overflow(n, c, &n) || __builtin_mul_overflow(n, d, &n) ||
        __builtin_mul_overflow(n, esize, &n) || n > MAX_EXTENT_BYTES)
        return -1;
    return n;
}

// [rows][heads][width] with (row, head) strides: heads must not overlap
// inside a row nor rows each other, in either nesting order of the strides.
struct Heads {
    int64_t st, sh, bytes;
};

inline conv_status check_heads(const int64_t *strides, int64_t rows, int64_t heads, int64_t width, int64_t esize,
                               bool output, Heads *h)
{
    h->st = strides ? strides[0] : heads * width;
    h->sh = strides ? strides[1] : width;
    if (h->st < 0 || h->sh < 0 || h->st > (int64_t(1) << 40) || h->sh > (int64_t(1) << 40))
        return CONV_ERR_LAYOUT;
    const bool heads_inner = (heads == 1 || h->sh >= width) && (rows <= 1 || h->st >= (heads - 1) * h->sh + width);
    const bool rows_inner = (rows <= 1 || h->st >= width) && (heads == 1 || h->sh >= (rows - 1) * h->st + width);
    if (output && !heads_inner && !rows_inner)
        return CONV_ERR_LAYOUT;
    if (rows == 0) {
        h->bytes = 0;
        return CONV_OK;
    }
    int64_t a, b, n;
    if (__builtin_mul_overflow(rows - 1, h->st, &a) || __builtin_mul_overflow(heads - 1, h->sh, &b) ||
        __builtin_add_overflow(a, b, &n) || __builtin_add_overflow(n, width, &n) ||
        __builtin_mul_overflow(n, esize, &n) || n > MAX_EXTENT_BYTES)
        return CONV_ERR_LAYOUT;
    h->bytes = n;
    return CONV_OK;
}

inline conv_status check_sequences(const int32_t *offsets, const void *state_in, const void *state_out,
                                   const int32_t *slots, int num_slots, int64_t tokens, int num_seqs,
                                   int64_t state_bytes, Sequences *s)
{
    if (num_seqs <= 0 || tokens < 0)
        return CONV_ERR_NONPOSITIVE;
    if (tokens > MAX_ROWS || num_seqs > MAX_ROWS)
        return CONV_ERR_UNSUPPORTED;
    if (!offsets && tokens % num_seqs != 0)
        return CONV_ERR_SHAPE;
    if (!aligned(offsets, 4) || !aligned(slots, 4))
        return CONV_ERR_LAYOUT;
    if (state_in || state_out) {
        if (num_slots <= 0)
            return CONV_ERR_NONPOSITIVE;
        if (!slots && num_slots < num_seqs)
            return CONV_ERR_SHAPE;
        if (state_in && state_out && state_in != state_out &&
            overlaps(flat_range(state_in, state_bytes), flat_range(state_out, state_bytes)))
            return CONV_ERR_ALIAS;
    }
    s->offsets = offsets;
    s->slots = slots;
    s->num_slots = num_slots;
    s->num_seqs = num_seqs;
    s->tokens = tokens;
    s->each = tokens / num_seqs;
    return CONV_OK;
}

// Whether an output range overlaps any of `n` others (empty ranges overlap
// nothing).
inline bool hits(Range out, const Range *others, int n)
{
    if (out.lo == out.hi)
        return false;
    for (int i = 0; i < n; ++i)
        if (others[i].lo != others[i].hi && overlaps(out, others[i]))
            return true;
    return false;
}

inline Range range_of(const void *p, int64_t bytes) { return p ? flat_range(p, bytes) : Range{0, 0}; }

}  // namespace convfwd
