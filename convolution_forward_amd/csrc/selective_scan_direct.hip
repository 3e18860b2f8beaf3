// The selective scan with a decay for each channel and state, token by token.
//
//   d = step(dt + bias);  h[n] = exp(d a[c,n]) h[n] + d x b[n]
//   y = (sum_n c[n] h[n] + skip x) silu(gate)
//
// A lane holds four states of one channel, LN lanes a channel (four times LN
// covers the states), a wave 64 / LN neighbouring channels: its states are
// one run of memory, and y is an exchange between LN lanes. No wave waits for
// another.
//
// Single tokens: the states' bytes are the time, each read and written once.
// Longer sequences are the chain from token to token; the next token's inputs
// are loaded a token ahead.
#include "common.h"
#include "eight_bit.h"
#include "internal.h"
#include "lanes.h"
#include "scan_math.h"
#include "sequences.h"

namespace convfwd {
namespace {

// One token's inputs as they lie in memory.
template <class T>
struct Token {
    T b[4] __attribute__((aligned(16))), c[4] __attribute__((aligned(16)));
    T x, dt, gate;
};

// WIDE: states, b and c allow pieces of four (a host rule).
template <class T, int LN, bool WIDE>
__global__ __launch_bounds__(256) void scan_direct_kernel(ScanProblem p, int slices)
{
    constexpr int CH = 64 / LN;
    const int lane = threadIdx.x & 63;
    const int64_t job = (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
    const int n = (int)(job / slices);
    if (n >= p.seq.num_seqs)
        return;
    const int c = (int)(job % slices) * CH + lane / LN, at = 4 * (lane % LN);
    const bool live = c < p.channels;       // lanes past the channels take the last one's inputs and store nothing
    const int ch = live ? c : p.channels - 1;
    const int group = ch / (p.channels / p.groups);
    const int64_t begin = seq_begin(p.seq, n), end = seq_begin(p.seq, n + 1);
    const int slot = p.state_in || p.state_out ? seq_slot(p.seq, n) : -1;
    const int64_t sat = ((int64_t)slot * p.channels + ch) * p.N + at;

    float h[4], a[4];
    const float *ap = p.a + (int64_t)ch * p.N + at;
    const bool held = p.state_in && slot >= 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = a[i] = 0.f;
    if constexpr (WIDE) {
        if (at < p.N) {
            const float4 v = *reinterpret_cast<const float4 *>(ap);
            a[0] = v.x, a[1] = v.y, a[2] = v.z, a[3] = v.w;
            if (held) {
                const float4 s = *reinterpret_cast<const float4 *>(p.state_in + sat);
                h[0] = s.x, h[1] = s.y, h[2] = s.z, h[3] = s.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at + i < p.N) {
                a[i] = ap[i];
                if (held)
                    h[i] = p.state_in[sat + i];
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a[i] *= LOG2E;
    const float skip = p.skip ? p.skip[ch] : 0.f, bias = p.bias ? p.bias[ch] : 0.f;
    const T *xp = static_cast<const T *>(p.x) + begin * p.xs + ch;
    const T *dp = static_cast<const T *>(p.dt) + begin * p.dts + ch;
    const T *gp = p.gate ? static_cast<const T *>(p.gate) + begin * p.gs + ch : nullptr;
    const T *bp = static_cast<const T *>(p.b) + begin * p.bst + group * p.bsg;
    const T *cp = static_cast<const T *>(p.c) + begin * p.cst + group * p.csg;
    T *yp = static_cast<T *>(p.y) + begin * p.ys + ch;

    auto load = [&](Token<T> &t) __attribute__((always_inline)) {
        t.x = *xp;
        t.dt = *dp;
        if (gp)
            t.gate = *gp;
        if constexpr (WIDE) {
            const int n0 = at < p.N ? at : 0;
            __builtin_memcpy(t.b, __builtin_assume_aligned(bp + n0, 4 * sizeof(T)), sizeof(t.b));
            __builtin_memcpy(t.c, __builtin_assume_aligned(cp + n0, 4 * sizeof(T)), sizeof(t.c));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n0 = at + i < p.N ? at + i : 0;
                t.b[i] = bp[n0];
                t.c[i] = cp[n0];
            }
        }
    };
    auto advance = [&]() __attribute__((always_inline)) {
        xp += p.xs;
        dp += p.dts;
        if (gp)
            gp += p.gs;
        bp += p.bst;
        cp += p.cst;
    };
    auto step = [&](const Token<T> &t) __attribute__((always_inline)) {
        const float x = load_as_f32(&t.x);
        const float d = step_size(load_as_f32(&t.dt) + bias, p.softplus);
        const float dx = d * x;
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = WIDE ? at < p.N : at + i < p.N;
            // States past the last one stay zeros, whatever x is.
            h[i] = in ? fmaf(__builtin_amdgcn_exp2f(d * a[i]), h[i], dx * load_as_f32(&t.b[i])) : 0.f;
            y = in ? fmaf(h[i], load_as_f32(&t.c[i]), y) : y;
        }
        y = lanes_sum<LN>(y);
        y = fmaf(skip, x, y);
        if (gp)
            y *= silu(load_as_f32(&t.gate));
        if (live && at == 0)
            store_rne(yp, y);
        yp += p.ys;
    };
    int64_t left = end - begin;
    if (left > 0) {
        Token<T> t0, t1;
        load(t0);
        for (; left > 2; left -= 2) {
            advance();
            load(t1);
            step(t0);
            advance();
            load(t0);
            step(t1);
        }
        if (left == 2) {
            advance();
            load(t1);
            step(t0);
            step(t1);
        } else {
            step(t0);
        }
    }
    if (p.state_out && slot >= 0 && live) {
        if constexpr (WIDE) {
            if (at < p.N)
                *reinterpret_cast<float4 *>(p.state_out + sat) = make_float4(h[0], h[1], h[2], h[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (at + i < p.N)
                    p.state_out[sat + i] = h[i];
        }
    }
}

int lanes_for(int N)
{
    int l = 1;
    while (4 * l < N)
        l *= 2;
    return l;
}

template <class T, int LN>
void launch_lanes(const ScanProblem &p, hipStream_t s)
{
    const int slices = (p.channels + 64 / LN - 1) / (64 / LN);
    const int64_t jobs = (int64_t)p.seq.num_seqs * slices;
    const int waves = jobs <= 1024 ? 1 : 4;     // few waves: one a workgroup, so that they spread over the compute units
    const dim3 grid((unsigned)((jobs + waves - 1) / waves)), block(64 * waves);
    const uintptr_t bc = (uintptr_t)p.b | (uintptr_t)p.c | (uintptr_t)((p.bst | p.bsg | p.cst | p.csg) * (int64_t)sizeof(T));
    const uintptr_t st = (uintptr_t)p.state_in | (uintptr_t)p.state_out | (uintptr_t)p.a;
    if (bc % (4 * sizeof(T)) == 0 && st % 16 == 0 && p.N % 4 == 0)
        hipLaunchKernelGGL((scan_direct_kernel<T, LN, true>), grid, block, 0, s, p, slices);
    else
        hipLaunchKernelGGL((scan_direct_kernel<T, LN, false>), grid, block, 0, s, p, slices);
}

template <class T>
void launch(const ScanProblem &p, hipStream_t s)
{
    switch (lanes_for(p.N)) {
    case 1: launch_lanes<T, 1>(p, s); break;
    case 2: launch_lanes<T, 2>(p, s); break;
    case 4: launch_lanes<T, 4>(p, s); break;
    case 8: launch_lanes<T, 8>(p, s); break;
    case 16: launch_lanes<T, 16>(p, s); break;
    case 32: launch_lanes<T, 32>(p, s); break;
    default: launch_lanes<T, 64>(p, s); break;
    }
}

}  // namespace

// The grid's threads stay below 2^32 (64 a wave, up to three waves idle).
bool scan_direct_supports(int num_seqs, int channels, int N)
{
    if (N > 256)
        return false;
    const int ch = 64 / lanes_for(N);
    return (int64_t)num_seqs * ((channels + ch - 1) / ch) <= (int64_t(1) << 26) - 4;
}

hipError_t launch_scan_direct(const ScanProblem &p, hipStream_t s)
{
    if (p.dtype == CONV_BF16)
        launch<uint16_t>(p, s);
    else
        launch<float>(p, s);
    return hipGetLastError();
}

}  // namespace convfwd
