// RMS norm with the residual's addition and an output in 8 bits.
//
//   h = x + r rounded to the tensors' type;  y_j = h_j * rsqrt(mean(h^2) + eps) * w_j
//   scale = max|y| / QMAX;  q = y / scale to nearest even
//
// One workgroup a row. The mean, the norm and the scale are fp32.
#include "common.h"
#include "eight_bit.h"
#include "internal.h"

namespace convfwd {
namespace {

constexpr int NT = 256;

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v += __shfl_xor(v, d);
    return v;
}

// The largest magnitude as bits: those of a NaN are above infinity's and
// infinity's above every number's, so nothing that is not finite is lost.
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v = max(v, (uint32_t)__shfl_xor((int)v, d));
    return v;
}

template <class T, bool E4M3>
__global__ __launch_bounds__(NT) void rms_norm_q8_kernel(NormProblem p)
{
    __shared__ float part[NT / 64];
    __shared__ uint32_t tops[NT / 64];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.xs;
    const T *r = p.residual ? static_cast<const T *>(p.residual) + row * p.rs : nullptr;
    const T *w = static_cast<const T *>(p.weight);
    T *h = p.h ? static_cast<T *>(p.h) + row * p.hs : nullptr;
    uint8_t *q = static_cast<uint8_t *>(p.q) + row * p.qs;
    float sum = 0.f;
    for (int j = threadIdx.x; j < p.width; j += NT) {
        float v = load_as_f32(x + j);
        if (r) {
            T t;
            store_from_f32(&t, v + load_as_f32(r + j));
            h[j] = t;
            v = load_as_f32(&t);
        }
        sum += v * v;
    }
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = 0.f;
    for (int i = 0; i < NT / 64; ++i)
        sum += part[i];
    const float rinv = 1.f / sqrtf(sum / (float)p.width + p.eps);
    const T *src = r ? h : x;
    uint32_t top_bits = 0;
    for (int j = threadIdx.x; j < p.width; j += NT)
        top_bits = max(top_bits, __float_as_uint(fabsf(load_as_f32(src + j) * rinv * load_as_f32(w + j))));
    top_bits = wave_max(top_bits);
    if ((threadIdx.x & 63) == 0)
        tops[threadIdx.x >> 6] = top_bits;
    __syncthreads();
    for (int i = 0; i < NT / 64; ++i)
        top_bits = max(top_bits, tops[i]);
    const float top = __uint_as_float(top_bits);
    constexpr float QMAX = E4M3 ? 448.f : 127.f;
    const bool fine = sum < INFINITY && top < INFINITY;
    const float inv = fine && top > 0.f ? QMAX / top : 0.f;
    if (threadIdx.x == 0)
        p.scale[row] = fine ? top / QMAX : NAN;
    for (int j = threadIdx.x; j < p.width; j += NT)
        q[j] = fine ? to_eight<E4M3>(load_as_f32(src + j) * rinv * load_as_f32(w + j) * inv) : 0;
}

template <class T>
void launch(const NormProblem &p, hipStream_t s)
{
    if (p.qdt == CONV_E4M3)
        hipLaunchKernelGGL((rms_norm_q8_kernel<T, true>), dim3((unsigned)p.rows), dim3(NT), 0, s, p);
    else
        hipLaunchKernelGGL((rms_norm_q8_kernel<T, false>), dim3((unsigned)p.rows), dim3(NT), 0, s, p);
}

}  // namespace

hipError_t launch_rms_norm_q8(const NormProblem &p, hipStream_t s)
{
    if (p.dtype == CONV_BF16)
        launch<uint16_t>(p, s);
    else
        launch<float>(p, s);
    return hipGetLastError();
}

}  // namespace convfwd
