// The selective scan with a decay for each channel and state, token by token.
//
//   d = step(dt + bias);  h[n] = exp(d a[c,n]) h[n] + d x b[n]
//   y = (sum_n c[n] h[n] + skip x) silu(gate)
//
// A lane holds four states of one channel or two, LN lanes a channel (four times
// LN covers the states), a wave 64 / LN neighbouring channels or twice as many:
// its states are one run of memory, and y is an exchange between LN lanes. No
// wave waits for another.
//
// Single tokens: the states' bytes are the time, each read once and written once,
// past the caches. 64 sequences of 8192 channels of 16 states, bf16: 16.1 us, 4.5
// TB/s, where the states lie in the last cache (16.9 with stores that stay in the
// caches), and 18.5 where they do not; 256: 62.5 us, 4.6 TB/s; one: 3.2 us, a
// launch. The offsets come first, one after the other, then the state and the
// rates, and the token's inputs last: that chain is what 64 sequences do not hide.
// Longer sequences are the chain from token to token; the next token's inputs
// are loaded a token ahead (64 of 8 tokens: 41 us; one of 1000 tokens of 2048
// channels of 64 states, more than tiles take: 419).
#include "common.h"
#include "eight_bit.h"
#include "internal.h"
#include "lanes.h"
#include "scan_math.h"
#include "sequences.h"

namespace convfwd {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// One token's inputs as they lie in memory, R channels a lane.
template <class T, int R>
struct Token {
    T b[4] __attribute__((aligned(16))), c[4] __attribute__((aligned(16)));
    T x[R], dt[R], gate[R];
};

// WIDE: states, b and c allow pieces of four, which R = 2 needs, as well as groups of whole slices (a host rule).
template <class T, int LN, int R, bool WIDE>
__global__ __launch_bounds__(256) void scan_direct_kernel(ScanProblem p, int slices)
{
    constexpr int CH = 64 / LN;
    const int lane = threadIdx.x & 63;
    // (The same in all lanes, which the compiler has to be told; below 2^26.)
    const uint32_t job = __builtin_amdgcn_readfirstlane(blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6));
    const int n = (int)(job / (uint32_t)slices);
    if (n >= p.seq.num_seqs)
        return;
    const int c0 = (int)(job % (uint32_t)slices) * CH * R + lane / LN, at = 4 * (lane % LN);
    const int64_t begin = seq_begin(p.seq, n), end = seq_begin(p.seq, n + 1);
    const int slot = p.state_in || p.state_out ? seq_slot(p.seq, n) : -1;

    int ch[R];              // lanes past the channels take the last one's inputs and store nothing
    bool live[R];
    float h[R][4], a[R][4], skip[R], bias[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        live[j] = c0 + j * CH < p.channels;
        ch[j] = live[j] ? c0 + j * CH : p.channels - 1;
    }
    int group = ch[0] / (p.channels / p.groups);
    if constexpr (R == 2)
        group = __builtin_amdgcn_readfirstlane(group);
    auto four = [&](float (&v)[4], const float *s) __attribute__((always_inline)) {
        if constexpr (WIDE) {
            if (at < p.N) {
                const f32x4 f = *reinterpret_cast<const f32x4 *>(s);
                v[0] = f[0], v[1] = f[1], v[2] = f[2], v[3] = f[3];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (at + i < p.N)
                    v[i] = s[i];
        }
    };
    auto place = [&](int j) __attribute__((always_inline)) { return (int64_t)ch[j] * p.N + at; };
    const int64_t sat = (int64_t)slot * p.channels * p.N;
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[j][i] = a[j][i] = 0.f;
    if (p.state_in && slot >= 0)
#pragma unroll
        for (int j = 0; j < R; ++j)
            four(h[j], p.state_in + sat + place(j));
#pragma unroll
    for (int j = 0; j < R; ++j) {
        four(a[j], p.a + place(j));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            a[j][i] = rate_of_log2(a[j][i]);
        skip[j] = p.skip ? p.skip[ch[j]] : 0.f;
        bias[j] = p.bias ? p.bias[ch[j]] : 0.f;
    }
    const T *xp = static_cast<const T *>(p.x) + begin * p.xs;
    const T *dp = static_cast<const T *>(p.dt) + begin * p.dts;
    const T *gp = p.gate ? static_cast<const T *>(p.gate) + begin * p.gs : nullptr;
    const T *bp = static_cast<const T *>(p.b) + begin * p.bst + group * p.bsg;
    const T *cp = static_cast<const T *>(p.c) + begin * p.cst + group * p.csg;
    T *yp = static_cast<T *>(p.y) + begin * p.ys;

    auto load = [&](Token<T, R> &t) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            t.x[j] = xp[ch[j]];
            t.dt[j] = dp[ch[j]];
            if (gp)
                t.gate[j] = gp[ch[j]];
        }
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
    auto step = [&](const Token<T, R> &t) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const float x = load_as_f32(&t.x[j]);
            const float d = step_size(load_as_f32(&t.dt[j]) + bias[j], p.softplus);
            const float dx = d * x;
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool in = WIDE ? at < p.N : at + i < p.N;
                // States past the last one stay zeros, whatever x is.
                h[j][i] = in ? fmaf(__builtin_amdgcn_exp2f(d * a[j][i]), h[j][i], dx * load_as_f32(&t.b[i])) : 0.f;
                y = in ? fmaf(h[j][i], load_as_f32(&t.c[i]), y) : y;
            }
            y = lanes_sum<LN>(y);
            y = fmaf(skip[j], x, y);
            if (gp)
                y *= silu(load_as_f32(&t.gate[j]));
            if (live[j] && at == 0)
                store_rne(yp + ch[j], y);
        }
        yp += p.ys;
    };
    int64_t left = end - begin;
    if (left > 0) {
        Token<T, R> t0, t1;
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
    if (p.state_out && slot >= 0) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float *const to = p.state_out + sat + place(j);
            if (!live[j])
                continue;
            if constexpr (WIDE) {
                if (at < p.N)
                    __builtin_nontemporal_store(f32x4{h[j][0], h[j][1], h[j][2], h[j][3]}, reinterpret_cast<f32x4 *>(to));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (at + i < p.N)
                        to[i] = h[j][i];
            }
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
    constexpr int CH = 64 / LN;
    const uintptr_t bc = (uintptr_t)p.b | (uintptr_t)p.c | (uintptr_t)((p.bst | p.bsg | p.cst | p.csg) * (int64_t)sizeof(T));
    const uintptr_t st = (uintptr_t)p.state_in | (uintptr_t)p.state_out | (uintptr_t)p.a;
    const bool wide = bc % (4 * sizeof(T)) == 0 && st % 16 == 0 && p.N % 4 == 0;
    int slices = (p.channels + CH - 1) / CH;
    int64_t jobs = (int64_t)p.seq.num_seqs * slices;
    // Two channels a lane from 8192 waves on, as many as run at once: a single token of 8192 channels of 16 states in 256
    // sequences takes 62.5 us (one a lane: 66.3), in 64 17 (17), in 16 5.5 (6.0), but in 4 4.1 (3.6). Four a lane were
    // slower than one in 256: 157 registers.
    const bool two = wide && jobs >= 8192 && p.channels / p.groups % (2 * CH) == 0;
    if (two) {
        slices /= 2;
        jobs /= 2;
    }
    const int waves = jobs <= 1024 ? 1 : 4;     // few waves: one a workgroup, so that they spread over the compute units
    const dim3 grid((unsigned)((jobs + waves - 1) / waves)), block(64 * waves);
    if (two)
        hipLaunchKernelGGL((scan_direct_kernel<T, LN, 2, true>), grid, block, 0, s, p, slices);
    else if (wide)
        hipLaunchKernelGGL((scan_direct_kernel<T, LN, 1, true>), grid, block, 0, s, p, slices);
    else
        hipLaunchKernelGGL((scan_direct_kernel<T, LN, 1, false>), grid, block, 0, s, p, slices);
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
