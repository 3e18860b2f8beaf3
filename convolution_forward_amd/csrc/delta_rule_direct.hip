// The gated delta rule, token by token, in fp32.
//
//   S = exp(g) S;  u = beta (v - S^T k);  S = S + k u^T;  o = scale S^T q
//
// Columns of S are independent, so a wave owns all Dk rows of 32 of them and
// no wave ever waits for another: lane (r, c) = (lane / 8, lane % 8) holds
// rows r*R .. r*R + R-1 (R = Dk / 8 rounded up to 8, 16 or 32) of columns
// 4c .. 4c+3, and a sum over rows is R products in the lane and three
// exchanges between the eight row groups. Both products use the old state:
//   S_new^T q = exp(g) (S^T q) + (k.q) u,
// so one pass over the registers and one exchange serve S^T k and S^T q.
#include "common.h"
#include "internal.h"
#include "sequences.h"

namespace convfwd {
namespace {

constexpr float UNIT_EPS = 1e-6f;

// Sum over the eight row groups (lane bits 3 to 5).
__device__ __forceinline__ float rows_sum(float v)
{
    v += __shfl_xor(v, 8);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// WIDE: heads, columns and rows allow 16-byte pieces (a host rule): S by four
// columns, q and k by R rows at once.
template <class T, int R, bool WIDE>
__global__ __launch_bounds__(256) void delta_direct_kernel(DeltaProblem p, int slices)
{
    const int lane = threadIdx.x & 63;
    const int rg = lane >> 3, c = lane & 7;
    const int64_t job = (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
    const int slice = (int)(job % slices);
    const int64_t nh = job / slices;
    const int n = (int)(nh / p.Hv), h = (int)(nh % p.Hv);
    if (n >= p.seq.num_seqs)
        return;
    const int col = slice * 32 + c * 4, row = rg * R;
    const int kh = h / (p.Hv / p.Hk);
    const int64_t begin = seq_begin(p.seq, n);
    const int64_t end = seq_begin(p.seq, n + 1);
    const int slot = p.state_in || p.state_out ? seq_slot(p.seq, n) : -1;
    const int64_t sat = ((int64_t)slot * p.Hv + h) * p.Dk * p.Dv;

    float S[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            S[i][j] = 0.f;
    if (p.state_in && slot >= 0) {
        const float *si = p.state_in + sat + (int64_t)row * p.Dv + col;
        if constexpr (WIDE) {
            if (row < p.Dk && col < p.Dv) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float4 v = *reinterpret_cast<const float4 *>(si + (int64_t)i * p.Dv);
                    S[i][0] = v.x, S[i][1] = v.y, S[i][2] = v.z, S[i][3] = v.w;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (row + i < p.Dk && col + j < p.Dv)
                        S[i][j] = si[(int64_t)i * p.Dv + j];
        }
    }
    for (int64_t t = begin; t < end; ++t) {
        const T *kp = static_cast<const T *>(p.k) + t * p.kst + kh * p.ksh;
        const T *qp = static_cast<const T *>(p.q) + t * p.qst + kh * p.qsh;
        float k[R], q[R];
        float kk = 0.f, qq = 0.f, kq = 0.f;
        if constexpr (WIDE) {
            T kv[R] __attribute__((aligned(16))) = {}, qv[R] __attribute__((aligned(16))) = {};
            if (row < p.Dk) {
                __builtin_memcpy(kv, __builtin_assume_aligned(kp + row, 16), sizeof(kv));
                __builtin_memcpy(qv, __builtin_assume_aligned(qp + row, 16), sizeof(qv));
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                k[i] = load_as_f32(kv + i);
                q[i] = load_as_f32(qv + i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                k[i] = row + i < p.Dk ? load_as_f32(kp + row + i) : 0.f;
                q[i] = row + i < p.Dk ? load_as_f32(qp + row + i) : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            kk = fmaf(k[i], k[i], kk);
            qq = fmaf(q[i], q[i], qq);
            kq = fmaf(k[i], q[i], kq);
        }
        kk = rows_sum(kk);
        qq = rows_sum(qq);
        kq = rows_sum(kq);
        const float rk = p.normalize ? 1.f / sqrtf(kk + UNIT_EPS) : 1.f;
        const float rq = (p.normalize ? 1.f / sqrtf(qq + UNIT_EPS) : 1.f) * p.scale;
        const float decay = expf(p.g[t * p.Hv + h]), beta = p.beta[t * p.Hv + h];
        float sk[4], sq[4], u[4], o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                a = fmaf(S[i][j], k[i], a);
                b = fmaf(S[i][j], q[i], b);
            }
            sk[j] = rows_sum(a);
            sq[j] = rows_sum(b);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v = col + j < p.Dv
                                ? load_as_f32(static_cast<const T *>(p.v) + t * p.vst + h * p.vsh + col + j) : 0.f;
            u[j] = beta * (v - decay * rk * sk[j]) * rk;       // the factor that k needs, too
            o[j] = rq * (decay * sq[j] + kq * u[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                S[i][j] = fmaf(k[i], u[j], decay * S[i][j]);
            if (rg == 0 && col + j < p.Dv)
                store_from_f32(static_cast<T *>(p.o) + t * p.ost + h * p.osh + col + j, o[j]);
        }
    }
    if (p.state_out && slot >= 0) {
        float *so = p.state_out + sat + (int64_t)row * p.Dv + col;
        if constexpr (WIDE) {
            if (row < p.Dk && col < p.Dv) {
#pragma unroll
                for (int i = 0; i < R; ++i)
                    *reinterpret_cast<float4 *>(so + (int64_t)i * p.Dv) = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (row + i < p.Dk && col + j < p.Dv)
                        so[(int64_t)i * p.Dv + j] = S[i][j];
        }
    }
}

template <class T, int R>
void launch_rows(const DeltaProblem &p, hipStream_t s)
{
    const int slices = (p.Dv + 31) / 32;
    const int64_t jobs = (int64_t)p.seq.num_seqs * p.Hv * slices;
    // Few waves: one a workgroup, so that they spread over the compute units.
    const int waves = jobs <= 1024 ? 1 : 4;
    const dim3 grid((unsigned)((jobs + waves - 1) / waves)), block(64 * waves);
    const uintptr_t bits = (uintptr_t)p.q | (uintptr_t)p.k | (uintptr_t)p.state_in | (uintptr_t)p.state_out |
                           (uintptr_t)((p.qst | p.qsh | p.kst | p.ksh) * (int64_t)sizeof(T));
    if (bits % 16 == 0 && p.Dk % R == 0 && p.Dv % 4 == 0)
        hipLaunchKernelGGL((delta_direct_kernel<T, R, true>), grid, block, 0, s, p, slices);
    else
        hipLaunchKernelGGL((delta_direct_kernel<T, R, false>), grid, block, 0, s, p, slices);
}

template <class T>
void launch(const DeltaProblem &p, hipStream_t s)
{
    if (p.Dk <= 64)
        launch_rows<T, 8>(p, s);
    else if (p.Dk <= 128)
        launch_rows<T, 16>(p, s);
    else
        launch_rows<T, 32>(p, s);
}

}  // namespace

hipError_t launch_delta_direct(const DeltaProblem &p, hipStream_t s)
{
    if ((int64_t)p.seq.num_seqs * p.Hv * ((p.Dv + 31) / 32) > (int64_t(1) << 32))
        return hipErrorInvalidValue;
    if (p.dtype == CONV_BF16)
        launch<uint16_t>(p, s);
    else
        launch<float>(p, s);
    return hipGetLastError();
}

}  // namespace convfwd
