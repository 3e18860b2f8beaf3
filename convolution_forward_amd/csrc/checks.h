// Host-side argument checks shared by the C ABI files.
#pragma once

#include <stdint.h>

#include "internal.h"

namespace convfwd {

// Half-open byte range [lo, hi) touched by a tensor.
struct Range {
    uintptr_t lo, hi;
};

// Largest byte extent of a tensor the library addresses. Kernels form
// element and byte offsets as int64 sums of index * stride terms, each no
// larger than the extent, so every such sum stays far from overflow.
constexpr int64_t MAX_EXTENT_BYTES = int64_t(1) << 60;

inline Range flat_range(const void *base, int64_t bytes)
{
    uintptr_t lo = (uintptr_t)base;
    return Range{lo, lo + (uintptr_t)bytes};
}

inline bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

inline conv_status launched(hipError_t e)
{
    if (e != hipSuccess)
        return CONV_ERR_HIP;
    return hipGetLastError() == hipSuccess ? CONV_OK : CONV_ERR_HIP;
}

}  // namespace convfwd
