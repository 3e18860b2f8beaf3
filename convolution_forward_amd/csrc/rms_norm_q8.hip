// RMS norm with the residual's addition and an output in 8 bits.
//
//   h = x + r rounded to the tensors' type;  y_j = h_j * rsqrt(mean(h^2) + eps) * w_j
//   scale = max|y| / QMAX;  q = y / scale to nearest even
//
// One pass over memory: a row's h stays in registers from its load to its
// quantised store, between the two reductions (sum of squares, largest |y|).
// The bytes are the time, 16 a load: x and r in, h and q out. 16384x4096 bf16
// with a residual, 75-77 us: 0.47 GB at 6.2 TB/s (a plain copy: 5.5). Few rows
// are the latency of a load and two reductions: 4x2048, 3.8 us.
//
// The mean, the norm and the scale are fp32. Rows need no alignment: the
// loads and stores are unaligned ones, and the last piece of a row goes value
// by value.
#include "common.h"
#include "eight_bit.h"
#include "internal.h"

namespace convfwd {
namespace {

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

// Both reductions over the WPR waves of a row.
template <int WPR>
struct Reduce {
    float part[2][WPR > 1 ? WPR : 1];
    uint32_t tops[WPR > 1 ? WPR : 1];

    // `again`: the row's second sum.
    __device__ __forceinline__ float sum(float v, int wave, int again = 0)
    {
        v = wave_sum(v);
        if constexpr (WPR > 1) {
            if ((threadIdx.x & 63) == 0)
                part[again][wave] = v;
            __syncthreads();
            v = 0.f;
#pragma unroll
            for (int i = 0; i < WPR; ++i)
                v += part[again][i];
        }
        return v;
    }

    __device__ __forceinline__ uint32_t top(uint32_t v, int wave)
    {
        v = wave_max(v);
        if constexpr (WPR > 1) {
            if ((threadIdx.x & 63) == 0)
                tops[wave] = v;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < WPR; ++i)
                v = max(v, tops[i]);
        }
        return v;
    }
};

// A mean square this small (only an eps as small allows it) has lost bits
// below fp32's range: such rows are squared again, times 2^100.
constexpr float TINY = 0x1p-96f, LIFT = 0x1p100f;

__device__ __forceinline__ float mean_square(float sum, const NormProblem &p) { return sum / (float)p.width + p.eps; }
__device__ __forceinline__ float lifted_mean_square(float sum, const NormProblem &p)
{
    return sum / (float)p.width + p.eps * LIFT * LIFT;
}

// (A row of zeros without an eps stays zeros.)
__device__ __forceinline__ float root_inverse(float ms) { return ms == 0.f ? 0.f : 1.f / sqrtf(ms); }

// Writes the row's scale; y * lift * inv is what is rounded. lift is 1, or
// 2^100 where top is so small that QMAX / top would overflow.
struct Quant {
    bool fine;
    float lift, inv;
};

template <bool E4M3>
__device__ __forceinline__ Quant quant_scale(float sum, uint32_t top_bits, float *scale, bool first)
{
    constexpr float QMAX = E4M3 ? 448.f : 127.f;
    const float top = __uint_as_float(top_bits);
    Quant q;
    q.fine = sum < INFINITY && top < INFINITY;
    q.lift = top < 0x1p-100f ? 0x1p100f : 1.f;
    q.inv = q.fine && top > 0.f ? QMAX / (top * q.lift) : 0.f;
    if (first)
        *scale = q.fine ? top / QMAX : NAN;
    return q;
}

template <class T>
struct Piece {
    static constexpr int V = 16 / sizeof(T);
    T v[V];
};

// 16 bytes at any alignment.
typedef unsigned int any16 __attribute__((ext_vector_type(4), aligned(1)));

// STREAM: the streaming hint, for what this call reads once (16384x4096, all
// three with it on loads and stores: 97 -> 77 us).
template <bool STREAM, class T>
__device__ __forceinline__ Piece<T> load_piece(const T *p, int left)
{
    Piece<T> x = {};
    if (left >= Piece<T>::V) {
        any16 v;
        if constexpr (STREAM)
            v = __builtin_nontemporal_load(reinterpret_cast<const any16 *>(p));
        else
            v = *reinterpret_cast<const any16 *>(p);
        __builtin_memcpy(&x, &v, 16);
    } else {
#pragma unroll
        for (int i = 0; i < Piece<T>::V; ++i)
            if (i < left)
                x.v[i] = p[i];
    }
    return x;
}

template <class E, int V>
__device__ __forceinline__ void store_piece(E *p, const E (&x)[V], int left)
{
    if (left >= V) {
        typedef unsigned int words __attribute__((ext_vector_type(sizeof(x) / 4), aligned(1)));
        words v;
        __builtin_memcpy(&v, x, sizeof(x));
        __builtin_nontemporal_store(v, reinterpret_cast<words *>(p));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < left)
                p[i] = x[i];
    }
}

// WPR waves a row, NV pieces of 16 bytes a lane; one wave a row takes four
// rows a workgroup and needs no barrier.
template <class T, int WPR, int NV, bool RES, bool E4M3>
__global__ __launch_bounds__(WPR == 1 ? 256 : 64 * WPR) void rms_norm_q8_kernel(NormProblem p)
{
    constexpr int V = Piece<T>::V;
    __shared__ Reduce<WPR> red;
    const int wave = threadIdx.x >> 6;
    const int64_t row = WPR == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
    if (WPR == 1 && row >= p.rows)
        return;
    const int at = WPR == 1 ? (threadIdx.x & 63) : threadIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.xs;
    const T *w = static_cast<const T *>(p.weight);
    Piece<T> h[NV], r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        h[i] = load_piece<true>(x + (at + i * 64 * WPR) * V, p.width - (at + i * 64 * WPR) * V);
    if constexpr (RES) {
        const T *rp = static_cast<const T *>(p.residual) + row * p.rs;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            r[i] = load_piece<true>(rp + (at + i * 64 * WPR) * V, p.width - (at + i * 64 * WPR) * V);
    }
    float sum = 0.f, y[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if constexpr (RES)
                store_rne(&h[i].v[j], load_as_f32(&h[i].v[j]) + load_as_f32(&r[i].v[j]));
            y[i][j] = load_as_f32(&h[i].v[j]);
            sum = fmaf(y[i][j], y[i][j], sum);
        }
        if constexpr (RES)
            store_piece(static_cast<T *>(p.h) + row * p.hs + (at + i * 64 * WPR) * V, h[i].v,
                        p.width - (at + i * 64 * WPR) * V);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        r[i] = load_piece<false>(w + (at + i * 64 * WPR) * V, p.width - (at + i * 64 * WPR) * V);
    sum = red.sum(sum, wave);
    float ms = mean_square(sum, p);
    if (__builtin_expect(ms < TINY, 0)) {       // the same for all of the row's waves
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                y[i][j] *= LIFT;
                sum = fmaf(y[i][j], y[i][j], sum);
            }
        sum = red.sum(sum, wave, 1);
        ms = lifted_mean_square(sum, p);
    }
    const float rinv = root_inverse(ms);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            y[i][j] = y[i][j] * rinv * load_as_f32(&r[i].v[j]);
            top = max(top, __float_as_uint(fabsf(y[i][j])));
        }
    top = red.top(top, wave);
    const Quant z = quant_scale<E4M3>(sum, top, p.scale + row, at == 0);
    const float inv = z.inv;
    uint8_t *q = static_cast<uint8_t *>(p.q) + row * p.qs;
    if (z.lift != 1.f)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j)
                y[i][j] *= z.lift;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        uint8_t o[V] __attribute__((aligned(8)));
#pragma unroll
        for (int j = 0; j < V; j += 4)
            reinterpret_cast<uint32_t *>(o)[j / 4] =
                z.fine ? to_eight4<E4M3>(y[i][j] * inv, y[i][j + 1] * inv, y[i][j + 2] * inv, y[i][j + 3] * inv) : 0u;
        store_piece(q + (at + i * 64 * WPR) * V, o, p.width - (at + i * 64 * WPR) * V);
    }
}

// Rows past what registers hold: the row is read again for each step.
constexpr int LONG_WAVES = 16;

template <class T, bool E4M3>
__global__ __launch_bounds__(64 * LONG_WAVES) void rms_norm_q8_long_kernel(NormProblem p)
{
    constexpr int NT = 64 * LONG_WAVES;
    __shared__ Reduce<LONG_WAVES> red;
    const int wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.xs;
    const T *r = p.residual ? static_cast<const T *>(p.residual) + row * p.rs : nullptr;
    const T *w = static_cast<const T *>(p.weight);
    T *h = p.h ? static_cast<T *>(p.h) + row * p.hs : nullptr;
    float sum = 0.f;
    for (int j = threadIdx.x; j < p.width; j += NT) {
        T t = x[j];
        if (r) {
            store_rne(&t, load_as_f32(&t) + load_as_f32(r + j));
            h[j] = t;
        }
        const float v = load_as_f32(&t);
        sum = fmaf(v, v, sum);
    }
    sum = red.sum(sum, wave);
    const T *src = r ? h : x;               // each thread reads back what it wrote
    float ms = mean_square(sum, p), up = 1.f;
    if (ms < TINY) {
        up = LIFT;
        sum = 0.f;
        for (int j = threadIdx.x; j < p.width; j += NT) {
            const float v = load_as_f32(src + j) * up;
            sum = fmaf(v, v, sum);
        }
        sum = red.sum(sum, wave, 1);
        ms = lifted_mean_square(sum, p);
    }
    const float rinv = root_inverse(ms);
    uint32_t top = 0;
    for (int j = threadIdx.x; j < p.width; j += NT)
        top = max(top, __float_as_uint(fabsf(load_as_f32(src + j) * up * rinv * load_as_f32(w + j))));
    top = red.top(top, wave);
    const Quant z = quant_scale<E4M3>(sum, top, p.scale + row, threadIdx.x == 0);
    uint8_t *q = static_cast<uint8_t *>(p.q) + row * p.qs;
    for (int j = threadIdx.x; j < p.width; j += NT)
        q[j] = z.fine ? (uint8_t)to_eight4<E4M3>(load_as_f32(src + j) * up * rinv * load_as_f32(w + j) * z.lift * z.inv, 0.f, 0.f, 0.f) : 0;
}

template <class T, int WPR, int NV, bool E4M3>
void launch_held(const NormProblem &p, hipStream_t s)
{
    const unsigned grid = (unsigned)(WPR == 1 ? (p.rows + 3) / 4 : p.rows);
    const unsigned block = WPR == 1 ? 256 : 64 * WPR;
    if (p.residual)
        hipLaunchKernelGGL((rms_norm_q8_kernel<T, WPR, NV, true, E4M3>), dim3(grid), dim3(block), 0, s, p);
    else
        hipLaunchKernelGGL((rms_norm_q8_kernel<T, WPR, NV, false, E4M3>), dim3(grid), dim3(block), 0, s, p);
}

// One wave a row up to two pieces a lane (no barrier, and enough rows to fill
// the chip), else the fewest of 4, 8 and 16 waves that hold it in four:
// 16384x4096 bf16 took 126 us at eight pieces in one wave, 97 at two in four.
template <class T, bool E4M3>
void launch(const NormProblem &p, hipStream_t s)
{
    constexpr int V = Piece<T>::V;
    const int pieces = (p.width + 64 * V - 1) / (64 * V);       // of one wave
    if (pieces <= 1) {
        launch_held<T, 1, 1, E4M3>(p, s);
    } else if (pieces <= 2 && p.rows >= 4096) {
        launch_held<T, 1, 2, E4M3>(p, s);
    } else if (pieces <= 4) {
        launch_held<T, 4, 1, E4M3>(p, s);
    } else if (pieces <= 8) {
        launch_held<T, 4, 2, E4M3>(p, s);
    } else if (pieces <= 16) {
        launch_held<T, 4, 4, E4M3>(p, s);
    } else if (pieces <= 32) {
        launch_held<T, 8, 4, E4M3>(p, s);
    } else if (pieces <= 64) {
        launch_held<T, 16, 4, E4M3>(p, s);
    } else {
        hipLaunchKernelGGL((rms_norm_q8_long_kernel<T, E4M3>), dim3((unsigned)p.rows), dim3(64 * LONG_WAVES), 0, s, p);
    }
}

}  // namespace

hipError_t launch_rms_norm_q8(const NormProblem &all, hipStream_t s)
{
    // By 2^21 rows, so that a grid's threads stay below 2^32.
    const int64_t most = 1 << 21, e = all.dtype == CONV_BF16 ? 2 : 4;
    auto at = [](auto *t, int64_t bytes) { return t ? (decltype(t))((uintptr_t)t + bytes) : nullptr; };
    for (int64_t first = 0; first < all.rows; first += most) {
        NormProblem p = all;
        p.rows = all.rows - first < most ? all.rows - first : most;
        p.x = at(all.x, first * all.xs * e);
        p.residual = at(all.residual, first * all.rs * e);
        p.h = at(all.h, first * all.hs * e);
        p.q = at(all.q, first * all.qs);
        p.scale = all.scale + first;
        const bool e4m3 = p.qdt == CONV_E4M3;
        if (p.dtype == CONV_BF16)
            e4m3 ? launch<uint16_t, true>(p, s) : launch<uint16_t, false>(p, s);
        else
            e4m3 ? launch<float, true>(p, s) : launch<float, false>(p, s);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace convfwd
