// Product of 8-bit operands, one thread per output: any sizes, strides and
// alignment. The reference form of matmul_q8; it reads each operand byte by
// byte and is bound by those loads.
#include "common.h"
#include "eight_bit.h"
#include "internal.h"

namespace convfwd {
namespace {

template <bool E4M3, class Y>
__global__ __launch_bounds__(256) void matmul_q8_direct_kernel(MatmulQ8Problem p, int64_t total)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / p.N;
        const int n = (int)(i - m * p.N);
        const uint8_t *x = static_cast<const uint8_t *>(p.x) + m * p.xs;
        const uint8_t *w = static_cast<const uint8_t *>(p.w) + n * p.ws;
        float sum;
        if constexpr (E4M3) {
            sum = 0.f;
            for (int k = 0; k < p.K; ++k)
                sum = fmaf(e4m3_to_f32(x[k]), e4m3_to_f32(w[k]), sum);
        } else {
            int acc = 0;
            for (int k = 0; k < p.K; ++k)
                acc += (int)(int8_t)x[k] * (int)(int8_t)w[k];
            sum = (float)acc;
        }
        const float v = sum * p.xscale[m] * p.wscale[n] + (p.bias ? p.bias[n] : 0.f);
        store_from_f32(static_cast<Y *>(p.y) + m * p.ys + n, v);
    }
}

template <bool E4M3, class Y>
void launch(const MatmulQ8Problem &p, hipStream_t s)
{
    const int64_t total = p.M * p.N;
    hipLaunchKernelGGL((matmul_q8_direct_kernel<E4M3, Y>), dim3(grid_for(total, 256)), dim3(256), 0, s, p, total);
}

}  // namespace

hipError_t launch_matmul_q8_direct(const MatmulQ8Problem &p, hipStream_t s)
{
    const bool e = p.qdt == CONV_E4M3, b = p.ydt == CONV_BF16;
    if (e)
        b ? launch<true, uint16_t>(p, s) : launch<true, float>(p, s);
    else
        b ? launch<false, uint16_t>(p, s) : launch<false, float>(p, s);
    return hipGetLastError();
}

}  // namespace convfwd
