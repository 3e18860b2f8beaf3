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

// Sums of U values (2 or 4) over each aligned group of U lanes: lane u of the
// group gets the sum of the values u. 3 and 9 instructions, against 2 and 8 for
// all sums in all lanes.
template <int U>
__device__ __forceinline__ float lanes_scatter(const float (&v)[U], int lane)
{
    static_assert(U == 2 || U == 4, "pairs or fours");
    const bool odd = lane & 1;
    const float a = (odd ? v[1] : v[0]) + lane_moved<0xB1>(odd ? v[0] : v[1]);
    if constexpr (U == 2) {
        return a;
    } else {
        const float b = (odd ? v[3] : v[2]) + lane_moved<0xB1>(odd ? v[2] : v[3]);
        const bool upper = lane & 2;
        return (upper ? b : a) + lane_moved<0x4E>(upper ? a : b);
    }
}

}  // namespace convfwd
