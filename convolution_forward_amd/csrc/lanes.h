// Sums over neighbouring lanes without LDS.
#pragma once

#include "common.h"

namespace convfwd {

template <int CTRL>
__device__ __forceinline__ float lane_moved(float v)
{
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, false));
}

// Sum over each aligned group of L lanes (a power of two), in every lane of
// it, always in the same order. Lanes change places inside four, then mirrored
// in 8 and 16, then rows of 16 and 32 are swapped.
template <int L>
__device__ __forceinline__ float lanes_sum(float v)
{
    if constexpr (L >= 2)
        v += lane_moved<0xB1>(v);       // quad_perm 1,0,3,2
    if constexpr (L >= 4)
        v += lane_moved<0x4E>(v);       // quad_perm 2,3,0,1
    if constexpr (L >= 8)
        v += lane_moved<0x141>(v);      // row_half_mirror
    if constexpr (L >= 16)
        v += lane_moved<0x140>(v);      // row_mirror
    if constexpr (L >= 32) {
        const uint32_t a = __float_as_uint(v);
        const auto s = __builtin_amdgcn_permlane16_swap(a, a, false, false);
        v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    if constexpr (L >= 64) {
        const uint32_t a = __float_as_uint(v);
        const auto s = __builtin_amdgcn_permlane32_swap(a, a, false, false);
        v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    return v;
}

}  // namespace convfwd
