// C ABI of the rotary and selective scan operators: argument validation,
// variant choice and launch. As in api.cpp, every argument error is returned
// before the first HIP call, kernels go on the caller's stream, and nothing is
// allocated.
#include <stdint.h>

#include "mixer_checks.h"

using namespace convfwd;

namespace {

// Whether two outputs or inputs of [rows][heads][width] never meet. Their
// address ranges do where both are columns of one buffer of rows; with one row
// stride S and rows that stay within it, they are apart if they are so within
// a row.
bool apart(Range ra, const Heads &a, int64_t row_a, Range rb, const Heads &b, int64_t row_b, int64_t esize)
{
    if (!hits(ra, &rb, 1))
        return true;
    const int64_t S = a.st * esize;
    if (a.st != b.st || S <= 0 || row_a > S || row_b > S)
        return false;
    int64_t d = (int64_t)(rb.lo % (uintptr_t)S) - (int64_t)(ra.lo % (uintptr_t)S);
    if (d < 0)
        d += S;
    return d >= row_a && d + row_b <= S;
}

bool known_variant(int v) { return v == CONV_VARIANT_AUTO || v == CONV_VARIANT_DIRECT || v == CONV_VARIANT_TILED; }

// Sizes, dtype and variant of the scans. *tiled says which kernel runs.
conv_status check_scan_sizes(int64_t tokens, int num_seqs, int channels, int groups, int N, conv_dtype dtype, int variant,
                             bool *tiled)
{
    if (tokens < 0 || num_seqs <= 0 || channels <= 0 || groups <= 0 || N <= 0)
        return CONV_ERR_NONPOSITIVE;
    if (channels % groups != 0)
        return CONV_ERR_SHAPE;
    if (!is_float(dtype))
        return CONV_ERR_DTYPE;
    if (tokens > MAX_ROWS || num_seqs > MAX_ROWS || channels > (1 << 23) || N > 256 || !known_variant(variant))
        return CONV_ERR_UNSUPPORTED;
    const bool can = scan_tiled_supports(tokens, num_seqs, channels, groups, N);
    // Tokens a sequence, as the host knows them (the mean), from which tiles are
    // faster. A lone sequence of 8192 channels of 16 states takes 8.8 to 9.8 us by
    // tiles up to 64 tokens, and token by token 8.2 for 16 of them, 13.4 for 32.
    // Once there are more workgroups than run at once, 8 such sequences take 55 us
    // by tiles for 32 tokens and 57 for 64 (token by token 25 and 44), 64 take 426
    // and 452 (127 and 243); tiles are ahead from some 100 and 220 tokens. But one
    // long sequence among short ones is the time token by token (one of 4033 tokens
    // with 63 of one: 2110 us, by tiles 514), so less is asked for.
    const bool alone = (int64_t)num_seqs * channels * N <= 512 * 256;
    const int least = alone ? 16 : 48;
    *tiled = variant == CONV_VARIANT_TILED || (variant == CONV_VARIANT_AUTO && can && tokens > least * (int64_t)num_seqs);
    return (*tiled ? can : scan_direct_supports(num_seqs, channels, N)) ? CONV_OK : CONV_ERR_UNSUPPORTED;
}

conv_status check_heads_sizes(int64_t tokens, int num_seqs, int H, int P, int groups, int N, conv_dtype dtype, int variant,
                              bool *tiled)
{
    if (tokens < 0 || num_seqs <= 0 || H <= 0 || P <= 0 || groups <= 0 || N <= 0)
        return CONV_ERR_NONPOSITIVE;
    if (H % groups != 0)
        return CONV_ERR_SHAPE;
    if (!is_float(dtype))
        return CONV_ERR_DTYPE;
    if (tokens > MAX_ROWS || num_seqs > MAX_ROWS || H > 65535 || P > 65536 || N > 256 || !known_variant(variant))
        return CONV_ERR_UNSUPPORTED;
    const bool can = heads_chunked_supports(tokens, num_seqs, H, P, groups, N, dtype);
    // Tokens a sequence, as the host knows them (the mean), from which chunks
    // are faster. bf16, heads of 64 x 128: a lone sequence of 128 heads takes 13.2
    // us by chunks up to 32 tokens, and token by token 11.6 for 12 of them, 14.2
    // for 16; 8 such sequences 22 us (token by token 20 for 4 tokens, 24 for 6), 64
    // of them 147 and 157 (123 and 158). fp32, 32 heads of 64 x 64, where a chunk
    // costs more: 11.9 us alone (24 tokens one by one 9.9, 32 12.1), 64 sequences
    // 98 for 32 tokens and 114 for 64 (69 and 118, level at 60; a long sequence
    // among short ones gains by chunks, so less is asked for).
    const bool alone = (int64_t)num_seqs * H * P <= 16384;
    const int least = dtype == CONV_F32 ? (alone ? 24 : 44) : alone ? 12 : 6;
    *tiled = variant == CONV_VARIANT_TILED || (variant == CONV_VARIANT_AUTO && can && tokens > least * (int64_t)num_seqs);
    return (*tiled ? can : heads_direct_supports(num_seqs, H, P, N)) ? CONV_OK : CONV_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

conv_status conv_rotary_fwd(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                            const void *positions, int position_bits, const float *frequencies, const void *q_weight,
                            const void *k_weight, void *q_out, const int64_t *qo_strides, void *k_out,
                            const int64_t *ko_strides, int64_t tokens, int Hq, int Hk, int D, int rotated, float eps,
                            float scale, int interleaved, conv_dtype dtype, void *stream)
{
    if (!frequencies || (tokens != 0 && (!q || !q_out || !positions || (Hk != 0 && (!k || !k_out)))))
        return CONV_ERR_NULL;
    if (tokens < 0 || Hq <= 0 || Hk < 0 || D <= 0 || rotated <= 0)
        return CONV_ERR_NONPOSITIVE;
    if (rotated % 2 != 0 || rotated > D)
        return CONV_ERR_SHAPE;
    if (!is_float(dtype))
        return CONV_ERR_DTYPE;
    if ((position_bits != 32 && position_bits != 64) || Hq > 65535 || Hk > 65535 || !rotary_supports(tokens, Hq + Hk, D))
        return CONV_ERR_UNSUPPORTED;
    const int64_t e = size_of(dtype);
    Heads hq, hk = {0, 0, 0}, oq, ok = {0, 0, 0};
    if (check_heads(q_strides, tokens, Hq, D, e, false, &hq) != CONV_OK ||
        check_heads(qo_strides, tokens, Hq, D, e, true, &oq) != CONV_OK ||
        (Hk && check_heads(k_strides, tokens, Hk, D, e, false, &hk) != CONV_OK) ||
        (Hk && check_heads(ko_strides, tokens, Hk, D, e, true, &ok) != CONV_OK) || !aligned(q, e) || !aligned(q_out, e) ||
        (Hk && (!aligned(k, e) || !aligned(k_out, e))) || !aligned(q_weight, e) || !aligned(k_weight, e) ||
        !aligned(positions, position_bits / 8) || !aligned(frequencies, 4))
        return CONV_ERR_LAYOUT;
    const Range rq = range_of(q, hq.bytes), rk = Hk ? range_of(k, hk.bytes) : Range{0, 0};
    const Range wq = range_of(q_out, oq.bytes), wk = Hk ? range_of(k_out, ok.bytes) : Range{0, 0};
    const Range in[4] = {range_of(positions, tokens * (position_bits / 8)), range_of(frequencies, (int64_t)rotated * 2),
                         range_of(q_weight, (int64_t)D * e), range_of(Hk ? k_weight : nullptr, (int64_t)D * e)};
    auto row = [&](const Heads &h, int heads) { return ((heads - 1) * h.sh + D) * e; };
    // An output may be its own input: a head is read before it is written, by the same lanes.
    const bool own_q = q_out == q && oq.st == hq.st && oq.sh == hq.sh, own_k = k_out == k && ok.st == hk.st && ok.sh == hk.sh;
    if (hits(wq, in, 4) || hits(wk, in, 4) || (!own_q && hits(wq, &rq, 1)) || (!own_k && hits(wk, &rk, 1)) ||
        !apart(wq, oq, row(oq, Hq), rk, hk, row(hk, Hk), e) || !apart(wk, ok, row(ok, Hk), rq, hq, row(hq, Hq), e) ||
        !apart(wq, oq, row(oq, Hq), wk, ok, row(ok, Hk), e))
        return CONV_ERR_ALIAS;
    if (tokens == 0)
        return CONV_OK;
    RotaryProblem p;
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    p.qst = hq.st;
    p.qsh = hq.sh;
    p.kst = hk.st;
    p.ksh = hk.sh;
    p.qot = oq.st;
    p.qoh = oq.sh;
    p.kot = ok.st;
    p.koh = ok.sh;
    p.qweight = q_weight;
    p.kweight = Hk ? k_weight : nullptr;
    p.positions = positions;
    p.frequencies = frequencies;
    p.tokens = tokens;
    p.wide = position_bits == 64;
    p.Hq = Hq;
    p.Hk = Hk;
    p.D = D;
    p.rotated = rotated;
    p.interleaved = interleaved;
    p.eps = eps;
    p.scale = scale;
    p.dtype = dtype;
    return launched(launch_rotary(p, (hipStream_t)stream));
}

int64_t conv_selective_scan_workspace(int64_t tokens, int num_seqs, int channels, int groups, int N, conv_dtype dtype,
                                      int variant)
{
    bool tiled;
    if (check_scan_sizes(tokens, num_seqs, channels, groups, N, dtype, variant, &tiled) != CONV_OK)
        return -1;
    return tiled ? scan_tiled_workspace(tokens, num_seqs, channels, groups, N) : 0;
}

conv_status conv_selective_scan_fwd(const void *x, int64_t x_stride, const void *dt, int64_t dt_stride, const float *a,
                                    const void *b, const int64_t *b_strides, const void *c, const int64_t *c_strides,
                                    const float *skip, const void *gate, int64_t gate_stride, const float *dt_bias, void *y,
                                    int64_t y_stride, const int32_t *seq_offsets, const float *state_in,
                                    float *state_out, const int32_t *slots, int num_slots, void *workspace,
                                    int64_t workspace_bytes, int64_t tokens, int num_seqs, int channels, int groups, int N,
                                    int softplus, conv_dtype dtype, int variant, void *stream)
{
    if (!a || (tokens != 0 && (!x || !dt || !b || !c || !y)))
        return CONV_ERR_NULL;
    bool tiled;
    conv_status st = check_scan_sizes(tokens, num_seqs, channels, groups, N, dtype, variant, &tiled);
    if (st != CONV_OK)
        return st;
    const int64_t e = size_of(dtype);
    const int64_t sb = state_in || state_out ? flat_bytes(num_slots > 0 ? num_slots : 1, channels, N, 1, 4) : 0;
    const int64_t xb = rows_bytes(tokens, x_stride, channels, e), db = rows_bytes(tokens, dt_stride, channels, e);
    const int64_t gb = gate ? rows_bytes(tokens, gate_stride, channels, e) : 0, yb = rows_bytes(tokens, y_stride, channels, e);
    Heads hb, hc;
    if (x_stride < channels || dt_stride < channels || (gate && gate_stride < channels) || y_stride < channels || xb < 0 ||
        db < 0 || gb < 0 || yb < 0 || check_heads(b_strides, tokens, groups, N, e, false, &hb) != CONV_OK ||
        check_heads(c_strides, tokens, groups, N, e, false, &hc) != CONV_OK || sb < 0 || !aligned(x, e) || !aligned(dt, e) ||
        !aligned(a, 4) || !aligned(b, e) || !aligned(c, e) || !aligned(skip, 4) || !aligned(gate, e) || !aligned(dt_bias, 4) ||
        !aligned(y, e) || !aligned(state_in, 4) || !aligned(state_out, 4) || !aligned(workspace, 256))
        return CONV_ERR_LAYOUT;
    ScanProblem p;
    st = check_sequences(seq_offsets, state_in, state_out, slots, num_slots, tokens, num_seqs, sb, &p.seq);
    if (st != CONV_OK)
        return st;
    const int64_t need = conv_selective_scan_workspace(tokens, num_seqs, channels, groups, N, dtype, variant);
    if (need > 0 && !workspace)
        return CONV_ERR_NULL;
    if (workspace_bytes < need)
        return CONV_ERR_SHAPE;
    const Range in[10] = {range_of(x, xb), range_of(dt, db), range_of(a, (int64_t)channels * N * 4), range_of(b, hb.bytes),
                          range_of(c, hc.bytes), range_of(skip, (int64_t)channels * 4), range_of(gate, gb),
                          range_of(dt_bias, (int64_t)channels * 4), range_of(seq_offsets, ((int64_t)num_seqs + 1) * 4),
                          range_of(slots, (int64_t)num_seqs * 4)};
    const Range ri = range_of(state_in, sb);
    const Range out[3] = {range_of(y, yb), range_of(state_out, sb), range_of(workspace, need)};
    for (int i = 0; i < 3; ++i)
        if (hits(out[i], in, 10) || (i != 1 && hits(out[i], &ri, 1)) || hits(out[i], out + i + 1, 2 - i))
            return CONV_ERR_ALIAS;
    if (tokens == 0 && !state_out)
        return CONV_OK;
    p.x = x;
    p.dt = dt;
    p.b = b;
    p.c = c;
    p.gate = gate;
    p.a = a;
    p.skip = skip;
    p.bias = dt_bias;
    p.y = y;
    p.xs = x_stride;
    p.dts = dt_stride;
    p.gs = gate_stride;
    p.ys = y_stride;
    p.bst = hb.st;
    p.bsg = hb.sh;
    p.cst = hc.st;
    p.csg = hc.sh;
    p.state_in = state_in;
    p.state_out = state_out;
    p.workspace = workspace;
    p.channels = channels;
    p.groups = groups;
    p.N = N;
    p.softplus = softplus;
    p.dtype = dtype;
    return launched(tiled ? launch_scan_tiled(p, (hipStream_t)stream) : launch_scan_direct(p, (hipStream_t)stream));
}

int64_t conv_selective_scan_heads_workspace(int64_t tokens, int num_seqs, int H, int P, int groups, int N, conv_dtype dtype,
                                            int variant)
{
    bool tiled;
    if (check_heads_sizes(tokens, num_seqs, H, P, groups, N, dtype, variant, &tiled) != CONV_OK)
        return -1;
    return tiled ? heads_chunked_workspace(tokens, num_seqs, H, P, groups, N, dtype) : 0;
}

conv_status conv_selective_scan_heads_fwd(const void *x, const int64_t *x_strides, const void *dt, int64_t dt_stride,
                                          const float *a, const void *b, const int64_t *b_strides, const void *c,
                                          const int64_t *c_strides, const float *skip, const void *gate,
                                          const int64_t *gate_strides, const float *dt_bias, void *y,
                                          const int64_t *y_strides, const int32_t *seq_offsets, const float *state_in,
                                          float *state_out, const int32_t *slots, int num_slots, void *workspace,
                                          int64_t workspace_bytes, int64_t tokens, int num_seqs, int H, int P, int groups,
                                          int N, int softplus, conv_dtype dtype, int variant, void *stream)
{
    if (!a || (tokens != 0 && (!x || !dt || !b || !c || !y)))
        return CONV_ERR_NULL;
    bool tiled;
    conv_status st = check_heads_sizes(tokens, num_seqs, H, P, groups, N, dtype, variant, &tiled);
    if (st != CONV_OK)
        return st;
    const int64_t e = size_of(dtype);
    const int64_t sb = state_in || state_out ? flat_bytes(num_slots > 0 ? num_slots : 1, H, P, N, 4) : 0;
    const int64_t db = rows_bytes(tokens, dt_stride, H, e);
    Heads hx, hg = {0, 0, 0}, hy, hb, hc;
    if (dt_stride < H || db < 0 || check_heads(x_strides, tokens, H, P, e, false, &hx) != CONV_OK ||
        (gate && check_heads(gate_strides, tokens, H, P, e, false, &hg) != CONV_OK) ||
        check_heads(y_strides, tokens, H, P, e, true, &hy) != CONV_OK ||
        check_heads(b_strides, tokens, groups, N, e, false, &hb) != CONV_OK ||
        check_heads(c_strides, tokens, groups, N, e, false, &hc) != CONV_OK || sb < 0 || !aligned(x, e) || !aligned(dt, e) ||
        !aligned(a, 4) || !aligned(b, e) || !aligned(c, e) || !aligned(skip, 4) || !aligned(gate, e) || !aligned(dt_bias, 4) ||
        !aligned(y, e) || !aligned(state_in, 4) || !aligned(state_out, 4) || !aligned(workspace, 256))
        return CONV_ERR_LAYOUT;
    HeadScanProblem p;
    st = check_sequences(seq_offsets, state_in, state_out, slots, num_slots, tokens, num_seqs, sb, &p.seq);
    if (st != CONV_OK)
        return st;
    const int64_t need = conv_selective_scan_heads_workspace(tokens, num_seqs, H, P, groups, N, dtype, variant);
    if (need > 0 && !workspace)
        return CONV_ERR_NULL;
    if (workspace_bytes < need)
        return CONV_ERR_SHAPE;
    const Range in[10] = {range_of(x, hx.bytes), range_of(dt, db), range_of(a, (int64_t)H * 4), range_of(b, hb.bytes),
                          range_of(c, hc.bytes), range_of(skip, (int64_t)H * 4), range_of(gate, hg.bytes),
                          range_of(dt_bias, (int64_t)H * 4), range_of(seq_offsets, ((int64_t)num_seqs + 1) * 4),
                          range_of(slots, (int64_t)num_seqs * 4)};
    const Range ri = range_of(state_in, sb);
    const Range out[3] = {range_of(y, hy.bytes), range_of(state_out, sb), range_of(workspace, need)};
    for (int i = 0; i < 3; ++i)
        if (hits(out[i], in, 10) || (i != 1 && hits(out[i], &ri, 1)) || hits(out[i], out + i + 1, 2 - i))
            return CONV_ERR_ALIAS;
    if (tokens == 0 && !state_out)
        return CONV_OK;
    p.x = x;
    p.dt = dt;
    p.b = b;
    p.c = c;
    p.gate = gate;
    p.a = a;
    p.skip = skip;
    p.bias = dt_bias;
    p.y = y;
    p.xst = hx.st;
    p.xsh = hx.sh;
    p.gst = hg.st;
    p.gsh = hg.sh;
    p.yst = hy.st;
    p.ysh = hy.sh;
    p.dts = dt_stride;
    p.bst = hb.st;
    p.bsg = hb.sh;
    p.cst = hc.st;
    p.csg = hc.sh;
    p.state_in = state_in;
    p.state_out = state_out;
    p.workspace = workspace;
    p.H = H;
    p.P = P;
    p.groups = groups;
    p.N = N;
    p.softplus = softplus;
    p.dtype = dtype;
    return launched(tiled ? launch_heads_chunked(p, (hipStream_t)stream) : launch_heads_direct(p, (hipStream_t)stream));
}

}  // extern "C"
