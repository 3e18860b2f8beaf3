// What the two selective scans share: step sizes, gates and decays.
//
// Exponentials are the instruction's after a product with log2 e: its error,
// |x| 2^-24 of the value, is that of rounding x itself to fp32.
#pragma once

#include <float.h>

#include "common.h"

namespace convfwd {

constexpr float LOG2E = 1.44269504088896340736f;

// A rate, in units of log 2. What is below fp32's numbers, minus infinity too, is
// the lowest of them: it forgets the state at every token but one of step zero,
// where minus infinity would make a NaN of it.
__device__ __forceinline__ float rate_of_log2(float a)
{
    const float r = a * LOG2E;
    return r < -FLT_MAX ? -FLT_MAX : r;
}

// A step size: v, or log(1 + exp(v)). log(1 + e) of 0 <= e <= 1 is
// 2 atanh(s), s = e / (2 + e) <= 1/3, which keeps the relative precision that
// 1 + e would lose where e is small. atanh(s) / s as a polynomial in s^2 (its
// Chebyshev interpolation over 0 .. 1/9, off by 2^-27.8 at most).
__device__ __forceinline__ float step_size(float v, bool softplus)
{
    if (!softplus)
        return v;
    const float e = __builtin_amdgcn_exp2f(-LOG2E * fabsf(v));
    const float s = e * __builtin_amdgcn_rcpf(2.f + e), q = s * s;
    float t = 0.14078889f;
    t = fmaf(t, q, 0.13982579f);
    t = fmaf(t, q, 0.20012298f);
    t = fmaf(t, q, 0.33333161f);
    t = fmaf(t, q, 1.f);
    return fmaf(2.f * s, t, fmaxf(v, 0.f));
}

// v / (1 + exp(-v)); the reciprocal is the instruction's, within 1 ulp.
__device__ __forceinline__ float silu(float v)
{
    return v * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-LOG2E * v));
}

}  // namespace convfwd
