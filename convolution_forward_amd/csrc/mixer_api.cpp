// C ABI of the token-mixer operators: argument validation, variant choice and
// launch. As in api.cpp, every argument error is returned before the first
// HIP call, kernels go on the caller's stream, and nothing is allocated.
#include <stdint.h>

#include "mixer_checks.h"

using namespace convfwd;

namespace {

// Sizes, dtype and variant of the delta rule. *tiled says which kernel runs.
conv_status check_delta_sizes(int64_t tokens, int num_seqs, int Hk, int Hv, int Dk, int Dv, conv_dtype dtype,
                              int variant, bool *tiled)
{
    if (tokens < 0 || num_seqs <= 0 || Hk <= 0 || Hv <= 0 || Dk <= 0 || Dv <= 0)
        return CONV_ERR_NONPOSITIVE;
    if (Hv % Hk != 0)
        return CONV_ERR_SHAPE;
    if (!is_float(dtype))
        return CONV_ERR_DTYPE;
    if (tokens > MAX_ROWS || num_seqs > MAX_ROWS || Dk > 256 || Dv > 65536 || Hv > 65535)
        return CONV_ERR_UNSUPPORTED;
    const bool can = delta_chunked_supports(tokens, num_seqs, Hk, Hv, Dk, Dv);
    // Tokens a sequence, as the host knows them (the mean), from which chunks
    // are faster. A lone sequence of 32 heads of 128 x 128 takes 16 us by chunks
    // up to 64 tokens, and token by token 15.8 for 16 of them, 18.6 for 20; once
    // the chunks' workgroups share compute units, 8 such sequences take 38 us
    // (token by token 37 for 24 tokens, 47 for 32) and 64 take 220 (224 and 291).
    // In fp32, where a chunk costs more: 23 us alone (28 tokens one by one 23.6),
    // 59 for 8 sequences (48 tokens 62, 64 80), 372 to 407 for 64 (397, 520).
    const bool alone = (int64_t)num_seqs * Hv * ((Dv + 15) / 16) <= 256;
    const int least = dtype == CONV_F32 ? (alone ? 28 : 50) : alone ? 16 : 26;
    if (variant != CONV_VARIANT_AUTO && variant != CONV_VARIANT_DIRECT && variant != CONV_VARIANT_TILED)
        return CONV_ERR_UNSUPPORTED;
    *tiled = variant == CONV_VARIANT_TILED || (variant == CONV_VARIANT_AUTO && can && tokens > least * (int64_t)num_seqs);
    return (*tiled ? can : delta_direct_supports(tokens, num_seqs, Hv, Dk, Dv)) ? CONV_OK : CONV_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

conv_status conv_rms_norm_q8_fwd(const void *x, int64_t x_stride, const void *residual, int64_t r_stride,
                                 const void *weight, void *h, int64_t h_stride, void *q, int64_t q_stride, float *scale,
                                 int64_t rows, int width, float eps, conv_dtype dtype, conv_dtype q_dtype, void *stream)
{
    if (!weight || (rows != 0 && (!x || !q || !scale || (residual && !h))))
        return CONV_ERR_NULL;
    if (rows < 0 || width <= 0)
        return CONV_ERR_NONPOSITIVE;
    if (!is_float(dtype) || !is_eight(q_dtype))
        return CONV_ERR_DTYPE;
    if ((h && !residual) || rows > MAX_ROWS)
        return CONV_ERR_UNSUPPORTED;
    const int64_t e = size_of(dtype);
    if (x_stride < width || q_stride < width || (residual && (r_stride < width || h_stride < width)) || !aligned(x, e) ||
        !aligned(residual, e) || !aligned(weight, e) || !aligned(h, e) || !aligned(scale, 4))
        return CONV_ERR_LAYOUT;
    const int64_t xb = rows_bytes(rows, x_stride, width, e), qb = rows_bytes(rows, q_stride, width, 1);
    const int64_t rb = residual ? rows_bytes(rows, r_stride, width, e) : 0;
    const int64_t hb = residual ? rows_bytes(rows, h_stride, width, e) : 0;
    if (xb < 0 || qb < 0 || rb < 0 || hb < 0)
        return CONV_ERR_LAYOUT;
    const Range in[3] = {range_of(x, xb), range_of(residual, rb), range_of(weight, (int64_t)width * e)};
    const Range rh = range_of(h, hb), rq = range_of(q, qb), rs = range_of(scale, rows * 4);
    // h may be x or the residual itself: each value is read before it is written, by the same thread.
    const bool own_x = h == x && h_stride == x_stride, own_r = h == residual && h_stride == r_stride;
    if (hits(rq, in, 3) || hits(rs, in, 3) || hits(rq, &rh, 1) || hits(rs, &rh, 1) || hits(rq, &rs, 1) ||
        (!own_x && hits(rh, &in[0], 1)) || (!own_r && hits(rh, &in[1], 1)) || hits(rh, &in[2], 1))
        return CONV_ERR_ALIAS;
    if (rows == 0)
        return CONV_OK;
    const NormProblem p = {x, residual, weight, h, q, scale, x_stride, r_stride, h_stride, q_stride, rows, width, eps,
                           dtype, q_dtype};
    return launched(launch_rms_norm_q8(p, (hipStream_t)stream));
}

conv_status conv_matmul_q8_fwd(const void *x, int64_t x_stride, const float *x_scale, const void *w, int64_t w_stride,
                               const float *w_scale, const float *bias, void *y, int64_t y_stride, int64_t M, int N,
                               int K, conv_dtype q_dtype, conv_dtype y_dtype, int variant, void *stream)
{
    if (!w || !w_scale || (M != 0 && (!x || !x_scale || !y)))
        return CONV_ERR_NULL;
    if (M < 0 || N <= 0 || K <= 0)
        return CONV_ERR_NONPOSITIVE;
    if (!is_eight(q_dtype) || !is_float(y_dtype))
        return CONV_ERR_DTYPE;
    // 127 * 127 * K, and one lane's -128s, must fit 32 bits: K * 2^14 < 2^31.
    if (M > MAX_ROWS || (q_dtype == CONV_I8 && K > 131071))
        return CONV_ERR_UNSUPPORTED;
    if (variant != CONV_VARIANT_AUTO && variant != CONV_VARIANT_DIRECT && variant != CONV_VARIANT_TILED)
        return CONV_ERR_UNSUPPORTED;
    const int64_t e = size_of(y_dtype);
    if (x_stride < K || w_stride < K || y_stride < N || !aligned(x_scale, 4) || !aligned(w_scale, 4) ||
        !aligned(bias, 4) || !aligned(y, e))
        return CONV_ERR_LAYOUT;
    const int64_t xb = rows_bytes(M, x_stride, K, 1), wb = rows_bytes(N, w_stride, K, 1), yb = rows_bytes(M, y_stride, N, e);
    if (xb < 0 || wb < 0 || yb < 0)
        return CONV_ERR_LAYOUT;
    const Range in[5] = {range_of(x, xb), range_of(w, wb), range_of(x_scale, M * 4), range_of(w_scale, (int64_t)N * 4),
                         range_of(bias, (int64_t)N * 4)};
    if (hits(range_of(y, yb), in, 5))
        return CONV_ERR_ALIAS;
    if (M == 0)
        return CONV_OK;
    const MatmulQ8Problem p = {x, w, x_scale, w_scale, bias, y, x_stride, w_stride, y_stride, M, N, K, q_dtype, y_dtype};
    const bool tiled = matmul_q8_tiled_supports(p);
    if (variant == CONV_VARIANT_TILED && !tiled)
        return CONV_ERR_UNSUPPORTED;
    return launched(variant == CONV_VARIANT_DIRECT || !tiled ? launch_matmul_q8_direct(p, (hipStream_t)stream)
                                                             : launch_matmul_q8(p, (hipStream_t)stream));
}

conv_status conv_causal1d_fwd(const void *x, int64_t x_stride, const void *w, const float *bias, void *y,
                              int64_t y_stride, const int32_t *seq_offsets, const void *state_in, void *state_out,
                              const int32_t *slots, int num_slots, int64_t tokens, int num_seqs, int channels, int taps,
                              int silu, conv_dtype dtype, void *stream)
{
    if (!w || (tokens != 0 && (!x || !y)))
        return CONV_ERR_NULL;
    if (channels <= 0 || taps <= 0)
        return CONV_ERR_NONPOSITIVE;
    if (!is_float(dtype))
        return CONV_ERR_DTYPE;
    if (taps < 2 || taps > 8)
        return CONV_ERR_UNSUPPORTED;
    const int64_t e = size_of(dtype);
    const int64_t sb = state_in || state_out ? flat_bytes(num_slots > 0 ? num_slots : 1, taps - 1, channels, 1, e) : 0;
    if (x_stride < channels || y_stride < channels || !aligned(x, e) || !aligned(w, e) || !aligned(bias, 4) ||
        !aligned(y, e) || !aligned(state_in, e) || !aligned(state_out, e) || sb < 0)
        return CONV_ERR_LAYOUT;
    Causal1dProblem p;
    const conv_status st =
        check_sequences(seq_offsets, state_in, state_out, slots, num_slots, tokens, num_seqs, sb, &p.seq);
    if (st != CONV_OK)
        return st;
    const int64_t xb = rows_bytes(tokens, x_stride, channels, e), yb = rows_bytes(tokens, y_stride, channels, e);
    if (xb < 0 || yb < 0)
        return CONV_ERR_LAYOUT;
    const Range in[5] = {range_of(x, xb), range_of(w, (int64_t)channels * taps * e), range_of(bias, (int64_t)channels * 4),
                         range_of(seq_offsets, ((int64_t)num_seqs + 1) * 4), range_of(slots, (int64_t)num_seqs * 4)};
    const Range ri = range_of(state_in, sb), ro = range_of(state_out, sb), ry = range_of(y, yb);
    if (hits(ry, in, 5) || hits(ry, &ri, 1) || hits(ro, in, 5) || hits(ro, &ry, 1))
        return CONV_ERR_ALIAS;
    if (tokens == 0 && !state_out)
        return CONV_OK;
    p.x = x;
    p.w = w;
    p.bias = bias;
    p.y = y;
    p.xs = x_stride;
    p.ys = y_stride;
    p.state_in = state_in;
    p.state_out = state_out;
    p.channels = channels;
    p.taps = taps;
    p.silu = silu;
    p.dtype = dtype;
    if (!causal1d_supports(p))
        return CONV_ERR_UNSUPPORTED;
    return launched(launch_causal1d(p, (hipStream_t)stream));
}

int64_t conv_delta_rule_workspace(int64_t tokens, int num_seqs, int Hk, int Hv, int Dk, int Dv, conv_dtype dtype,
                                  int variant)
{
    bool tiled;
    if (check_delta_sizes(tokens, num_seqs, Hk, Hv, Dk, Dv, dtype, variant, &tiled) != CONV_OK)
        return -1;
    return tiled ? delta_chunked_workspace(tokens, num_seqs, Hk, Hv, Dk, dtype) : 0;
}

conv_status conv_delta_rule_fwd(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                                const void *v, const int64_t *v_strides, const float *g, const float *beta,
                                const int32_t *seq_offsets, const float *state_in, float *state_out,
                                const int32_t *slots, int num_slots, void *o, const int64_t *o_strides, void *workspace,
                                int64_t workspace_bytes, int64_t tokens, int num_seqs, int Hk, int Hv, int Dk, int Dv,
                                float scale, int normalize, conv_dtype dtype, int variant, void *stream)
{
    if (tokens != 0 && (!q || !k || !v || !g || !beta || !o))
        return CONV_ERR_NULL;
    bool tiled;
    conv_status st = check_delta_sizes(tokens, num_seqs, Hk, Hv, Dk, Dv, dtype, variant, &tiled);
    if (st != CONV_OK)
        return st;
    const int64_t e = size_of(dtype);
    const int64_t sb = state_in || state_out ? flat_bytes(num_slots > 0 ? num_slots : 1, Hv, Dk, Dv, 4) : 0;
    Heads hq, hk, hv, ho;
    if (check_heads(q_strides, tokens, Hk, Dk, e, false, &hq) != CONV_OK ||
        check_heads(k_strides, tokens, Hk, Dk, e, false, &hk) != CONV_OK ||
        check_heads(v_strides, tokens, Hv, Dv, e, false, &hv) != CONV_OK ||
        check_heads(o_strides, tokens, Hv, Dv, e, true, &ho) != CONV_OK || sb < 0 || !aligned(q, e) || !aligned(k, e) ||
        !aligned(v, e) || !aligned(o, e) || !aligned(g, 4) || !aligned(beta, 4) || !aligned(state_in, 4) ||
        !aligned(state_out, 4) || !aligned(workspace, 256))
        return CONV_ERR_LAYOUT;
    DeltaProblem p;
    st = check_sequences(seq_offsets, state_in, state_out, slots, num_slots, tokens, num_seqs, sb, &p.seq);
    if (st != CONV_OK)
        return st;
    const int64_t need = conv_delta_rule_workspace(tokens, num_seqs, Hk, Hv, Dk, Dv, dtype, variant);
    if (need > 0 && !workspace)
        return CONV_ERR_NULL;
    if (workspace_bytes < need)
        return CONV_ERR_SHAPE;
    const Range in[7] = {range_of(q, hq.bytes), range_of(k, hk.bytes), range_of(v, hv.bytes),
                         range_of(g, tokens * Hv * 4), range_of(beta, tokens * Hv * 4),
                         range_of(seq_offsets, ((int64_t)num_seqs + 1) * 4), range_of(slots, (int64_t)num_seqs * 4)};
    const Range ri = range_of(state_in, sb);
    const Range out[3] = {range_of(o, ho.bytes), range_of(state_out, sb), range_of(workspace, need)};
    for (int i = 0; i < 3; ++i)
        if (hits(out[i], in, 7) || (i != 1 && hits(out[i], &ri, 1)) || hits(out[i], out + i + 1, 2 - i))
            return CONV_ERR_ALIAS;
    if (tokens == 0 && !state_out)
        return CONV_OK;
    p.q = q;
    p.k = k;
    p.v = v;
    p.g = g;
    p.beta = beta;
    p.o = o;
    p.qst = hq.st;
    p.qsh = hq.sh;
    p.kst = hk.st;
    p.ksh = hk.sh;
    p.vst = hv.st;
    p.vsh = hv.sh;
    p.ost = ho.st;
    p.osh = ho.sh;
    p.state_in = state_in;
    p.state_out = state_out;
    p.workspace = workspace;
    p.Hk = Hk;
    p.Hv = Hv;
    p.Dk = Dk;
    p.Dv = Dv;
    p.scale = scale;
    p.normalize = normalize;
    p.dtype = dtype;
    return launched(tiled ? launch_delta_chunked(p, (hipStream_t)stream) : launch_delta_direct(p, (hipStream_t)stream));
}

}  // extern "C"
