// Rounding to 8-bit values and to bf16.
#pragma once

#include "common.h"

namespace convfwd {

__device__ __forceinline__ float e4m3_to_f32(uint8_t b) { return __builtin_amdgcn_cvt_f32_fp8((int)b, 0); }

// Four values as bytes, nearest even. |v| <= 127 (int8) or 448 (e4m3), up to a
// rounding that stays below the next value: no clamp. int8: adding 1.5 * 2^23
// leaves the rounded integer in a float's low bits.
template <bool E4M3>
__device__ __forceinline__ uint32_t to_eight4(float a, float b, float c, float d)
{
    if constexpr (E4M3) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
    } else {
        constexpr float M = 12582912.f;
        const uint32_t ab = __builtin_amdgcn_perm(__float_as_uint(b + M), __float_as_uint(a + M), 0x0c0c0400u);
        const uint32_t cd = __builtin_amdgcn_perm(__float_as_uint(d + M), __float_as_uint(c + M), 0x04000c0cu);
        return ab | cd;
    }
}

// The two narrow roundings as one conversion instruction each (nearest even).
__device__ __forceinline__ void store_rne(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_rne(uint16_t *p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

}  // namespace convfwd
