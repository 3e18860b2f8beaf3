// 8-bit values: rounding to them, and the reductions the norm needs.
#pragma once

#include "common.h"

namespace convfwd {

// e4m3 of a float in [-448, 448], nearest even (the conversion instruction
// works on pairs; the second is a zero).
__device__ __forceinline__ uint8_t f32_to_e4m3(float v)
{
    return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(v, 0.f, 0, false) & 0xff);
}

__device__ __forceinline__ float e4m3_to_f32(uint8_t b) { return __builtin_amdgcn_cvt_f32_fp8((int)b, 0); }

// Signed 8-bit integer of a float in [-127, 127], nearest even.
__device__ __forceinline__ uint8_t f32_to_i8(float v) { return (uint8_t)(int8_t)__float2int_rn(v); }

template <bool E4M3>
__device__ __forceinline__ uint8_t to_eight(float v)
{
    constexpr float top = E4M3 ? 448.f : 127.f;
    v = fminf(fmaxf(v, -top), top);
    return E4M3 ? f32_to_e4m3(v) : f32_to_i8(v);
}

}  // namespace convfwd
