// The gated delta rule, token by token, in fp32.
//
//   S = exp(g) S;  u = beta (v - S^T k);  S = S + k u^T;  o = scale S^T q
//
// Columns of S are independent, so a wave owns all Dk rows of 4 CL of them
// and no wave ever waits for another: lane (r, c) = (lane / CL, lane % CL)
// holds rows r*R .. r*R + R-1 of columns 4c .. 4c+3, and a sum over rows is R
// products in the lane and an exchange between the 64 / CL row groups (lane
// rotations and row swaps, no LDS). Both products use the old state:
//   S_new^T q = exp(g) (S^T q) + (k.q) u,
// so one pass over the registers and one exchange serve S^T k and S^T q.
//
// Single tokens: the state's bytes are the time. 32 columns a wave (whole
// 128-byte lines), every load of the state in flight at once. Longer
// sequences: the chain from token to token is, so the next token's inputs are
// loaded a token ahead and a wave takes 16 columns, half the work a step.
//
// 128 sequences of one token, 32 heads of 128 x 128: 99 us, 0.54 GB at 5.4
// TB/s; one sequence, 4.3 us. Long ones are their chain, 0.7 us a token
// (by chunks less from some 16 to 60 tokens on).
#include "common.h"
#include "eight_bit.h"
#include "internal.h"
#include "sequences.h"

namespace convfwd {
namespace {

constexpr float UNIT_EPS = 1e-6f;

template <int N>
__device__ __forceinline__ float rotated(float v)      // by N lanes within 16
{
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x120 + N, 0xf, 0xf, false));
}

// Sum over the row groups, in every lane.
template <int CL>
__device__ __forceinline__ float rows_sum(float v)
{
    if constexpr (CL <= 4)
        v += rotated<4>(v);
    v += rotated<8>(v);
    const uint32_t a = __float_as_uint(v);
    const auto s16 = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    v = __uint_as_float(s16[0]) + __uint_as_float(s16[1]);
    const uint32_t b = __float_as_uint(v);
    const auto s32 = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return __uint_as_float(s32[0]) + __uint_as_float(s32[1]);
}

// One token's inputs as they lie in memory.
template <class T, int R>
struct Token {
    T k[R] __attribute__((aligned(16))), q[R] __attribute__((aligned(16))), v[4] __attribute__((aligned(8)));
    float g, beta;
};

// WIDE: heads, columns and rows allow pieces of R rows and four columns (a
// host rule); rows and columns past the head then come in whole pieces.
template <class T, int R, int CL, bool WIDE>
__global__ __launch_bounds__(256) void delta_direct_kernel(DeltaProblem p, int slices)
{
    const int lane = threadIdx.x & 63;
    const int rg = lane / CL, c = lane % CL;
    const int64_t job = (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
    const int slice = (int)(job % slices);
    const int64_t nh = job / slices;
    const int n = (int)(nh / p.Hv), h = (int)(nh % p.Hv);
    if (n >= p.seq.num_seqs)
        return;
    const int col = (slice * CL + c) * 4, row = rg * R;
    const int kh = h / (p.Hv / p.Hk);
    const int64_t begin = seq_begin(p.seq, n);
    const int64_t end = seq_begin(p.seq, n + 1);
    const int slot = p.state_in || p.state_out ? seq_slot(p.seq, n) : -1;
    const int64_t sat = ((int64_t)slot * p.Hv + h) * p.Dk * p.Dv;
    const bool here = row < p.Dk && col < p.Dv;

    float S[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            S[i][j] = 0.f;
    if (p.state_in && slot >= 0 && here) {
        const float *si = p.state_in + sat + (int64_t)row * p.Dv + col;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if constexpr (WIDE) {
                const float4 v = *reinterpret_cast<const float4 *>(si + (int64_t)i * p.Dv);
                S[i][0] = v.x, S[i][1] = v.y, S[i][2] = v.z, S[i][3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (row + i < p.Dk && col + j < p.Dv)
                        S[i][j] = si[(int64_t)i * p.Dv + j];
            }
        }
    }
    // Lanes past the head take their inputs from its first row and column: their products meet zeros of S, and k and
    // q are zeroed below where they count.
    const T *kp = static_cast<const T *>(p.k) + begin * p.kst + kh * p.ksh;
    const T *qp = static_cast<const T *>(p.q) + begin * p.qst + kh * p.qsh;
    const T *vp = static_cast<const T *>(p.v) + begin * p.vst + h * p.vsh;
    const float *gp = p.g + begin * p.Hv + h, *bp = p.beta + begin * p.Hv + h;
    T *op = static_cast<T *>(p.o) + begin * p.ost + h * p.osh + col;
    auto load = [&](Token<T, R> &x) __attribute__((always_inline)) {
        if constexpr (WIDE) {
            const int at = row < p.Dk ? row : 0, vt = col < p.Dv ? col : 0;
            __builtin_memcpy(x.k, __builtin_assume_aligned(kp + at, R * sizeof(T) < 16 ? R * sizeof(T) : 16), sizeof(x.k));
            __builtin_memcpy(x.q, __builtin_assume_aligned(qp + at, R * sizeof(T) < 16 ? R * sizeof(T) : 16), sizeof(x.q));
            __builtin_memcpy(x.v, __builtin_assume_aligned(vp + vt, 4 * sizeof(T)), sizeof(x.v));
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int at = row + i < p.Dk ? row + i : 0;
                x.k[i] = kp[at];
                x.q[i] = qp[at];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x.v[j] = vp[col + j < p.Dv ? col + j : 0];
        }
        x.g = *gp;
        x.beta = *bp;
    };
    auto advance = [&]() __attribute__((always_inline)) {
        kp += p.kst;
        qp += p.qst;
        vp += p.vst;
        gp += p.Hv;
        bp += p.Hv;
    };
    auto step = [&](const Token<T, R> &x) __attribute__((always_inline)) {
        float k[R], q[R];
        float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const bool in = WIDE ? row < p.Dk : row + i < p.Dk;
            k[i] = in ? load_as_f32(&x.k[i]) : 0.f;
            q[i] = in ? load_as_f32(&x.q[i]) : 0.f;
            kk = fmaf(k[i], k[i], kk);
            qq = fmaf(q[i], q[i], qq);
            kq = fmaf(k[i], q[i], kq);
        }
        float rk = 1.f, rq = p.scale;
        if (p.normalize) {
            rk = __builtin_amdgcn_rsqf(rows_sum<CL>(kk) + UNIT_EPS);
            rq *= __builtin_amdgcn_rsqf(rows_sum<CL>(qq) + UNIT_EPS);
        }
        kq = rows_sum<CL>(kq);
        const float decay = __expf(x.g);        // off by |g| 2^-24 of it, and the roots above by 1 ulp
        float sk[4], sq[4], u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                a = fmaf(S[i][j], k[i], a);
                b = fmaf(S[i][j], q[i], b);
            }
            sk[j] = a;
            sq[j] = b;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sk[j] = rows_sum<CL>(sk[j]);
            sq[j] = rows_sum<CL>(sq[j]);
        }
        T o[4] __attribute__((aligned(16)));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u[j] = x.beta * (load_as_f32(&x.v[j]) - decay * rk * sk[j]) * rk;     // with the factor that k needs, too
            store_rne(&o[j], rq * (decay * sq[j] + kq * u[j]));
#pragma unroll
            for (int i = 0; i < R; ++i)
                S[i][j] = fmaf(k[i], u[j], decay * S[i][j]);
        }
        if (rg == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (col + j < p.Dv)
                    op[j] = o[j];
        }
        op += p.ost;
    };
    int64_t left = end - begin;
    if (left > 0) {
        Token<T, R> x0, x1;
        load(x0);
        for (; left > 2; left -= 2) {
            advance();
            load(x1);
            step(x0);
            advance();
            load(x0);
            step(x1);
        }
        if (left == 2) {
            advance();
            load(x1);
            step(x0);
            step(x1);
        } else {
            step(x0);
        }
    }
    if (p.state_out && slot >= 0 && here) {
        float *so = p.state_out + sat + (int64_t)row * p.Dv + col;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if constexpr (WIDE) {
                *reinterpret_cast<float4 *>(so + (int64_t)i * p.Dv) = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (row + i < p.Dk && col + j < p.Dv)
                        so[(int64_t)i * p.Dv + j] = S[i][j];
            }
        }
    }
}

template <class T, int R, int CL>
void launch_rows(const DeltaProblem &p, hipStream_t s)
{
    const int slices = (p.Dv + 4 * CL - 1) / (4 * CL);
    const int64_t jobs = (int64_t)p.seq.num_seqs * p.Hv * slices;
    // Few waves: one a workgroup, so that they spread over the compute units.
    // (Single tokens, one wave a workgroup against four: 128 waves 4.3 us
    // against 5.2, 512 6.9 against 7.2, 1024 9.9 against 9.6, 16384 106 against 101.)
    const int waves = jobs <= 512 ? 1 : 4;
    const dim3 grid((unsigned)((jobs + waves - 1) / waves)), block(64 * waves);
    const uintptr_t qk = (uintptr_t)p.q | (uintptr_t)p.k | (uintptr_t)((p.qst | p.qsh | p.kst | p.ksh) * (int64_t)sizeof(T));
    const uintptr_t v = (uintptr_t)p.v | (uintptr_t)((p.vst | p.vsh) * (int64_t)sizeof(T));
    const uintptr_t st = (uintptr_t)p.state_in | (uintptr_t)p.state_out;
    if (qk % 16 == 0 && v % (4 * sizeof(T)) == 0 && st % 16 == 0 && p.Dk % R == 0 && p.Dv % 4 == 0)
        hipLaunchKernelGGL((delta_direct_kernel<T, R, CL, true>), grid, block, 0, s, p, slices);
    else
        hipLaunchKernelGGL((delta_direct_kernel<T, R, CL, false>), grid, block, 0, s, p, slices);
}

bool single_tokens(int64_t tokens, int num_seqs) { return tokens <= 4 * (int64_t)num_seqs; }

template <class T>
void launch(const DeltaProblem &p, hipStream_t s)
{
    // 32 columns a wave against 16, 32 heads: one token 4.3 us against 5.2, of
    // 128 sequences 101 against 107; four tokens 7.3 either way; eight 11.1
    // against 9.9. (Past 128 rows the registers hold 16 columns a wave only.)
    const bool single = single_tokens(p.seq.tokens, p.seq.num_seqs);
    if (p.Dk <= 64)
        single ? launch_rows<T, 8, 8>(p, s) : launch_rows<T, 4, 4>(p, s);
    else if (p.Dk <= 128)
        single ? launch_rows<T, 16, 8>(p, s) : launch_rows<T, 8, 4>(p, s);
    else
        launch_rows<T, 16, 4>(p, s);
}

}  // namespace

// The grid's threads stay below 2^32 (64 a wave, up to three waves idle).
bool delta_direct_supports(int64_t tokens, int num_seqs, int Hv, int Dk, int Dv)
{
    const int columns = single_tokens(tokens, num_seqs) && Dk <= 128 ? 32 : 16;
    return (int64_t)num_seqs * Hv * ((Dv + columns - 1) / columns) <= (int64_t(1) << 26) - 4;
}

hipError_t launch_delta_direct(const DeltaProblem &p, hipStream_t s)
{
    if (p.dtype == CONV_BF16)
        launch<uint16_t>(p, s);
    else
        launch<float>(p, s);
    return hipGetLastError();
}

}  // namespace convfwd
