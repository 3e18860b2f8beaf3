// The selective scan with one decay a head, token by token.
//
//   d = step(dt + bias);  S = exp(d a) S + d x b^T;  y = (S c + skip x) silu(gate)
//
// Rows of S [P,N] are independent: eight lanes share a row, each with every
// eighth piece of four states, so that a load takes whole 128-byte lines of
// eight rows and y is an exchange between eight lanes. A wave owns 8 RL rows
// and waits for no other.
//
// Single tokens: the states' bytes are the time, each read and written once, past
// the caches. 128 sequences of 128 heads of 64 x 128, bf16: 173 us, 6.25 TB/s
// (through the caches 181); 8: 13.7; one: 4.3. fp32, where two tokens of b and c
// leave room for three waves a SIMD instead of four: 188. 129 to 256 states take
// 216 registers in bf16, two waves (64 sequences of 128 heads of 64 x 256, as
// many states: 187 us), and 278 in fp32, one wave (236).
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

typedef float f32x4 __attribute__((ext_vector_type(4)));

// One token's inputs as they lie in memory.
template <class T, int KV, int RL>
struct Token {
    T b[KV][4] __attribute__((aligned(16))), c[KV][4] __attribute__((aligned(16)));
    T x[RL], gate[RL], dt;
};

// KV pieces of 32 states. WIDE: states, b and c allow pieces of four (a host rule).
template <class T, int KV, int RL, bool WIDE>
__global__ __launch_bounds__(256) void heads_direct_kernel(HeadScanProblem p, int slices)
{
    const int lane = threadIdx.x & 63;
    const int row = lane >> 3, at = 4 * (lane & 7);
    // (The same in all lanes, which the compiler has to be told; below 2^26.)
    const uint32_t job = __builtin_amdgcn_readfirstlane(blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6));
    const uint32_t nh = job / (uint32_t)slices;
    const int slice = (int)(job % (uint32_t)slices), n = (int)(nh / (uint32_t)p.H), h = (int)(nh % (uint32_t)p.H);
    if (n >= p.seq.num_seqs)
        return;
    const int group = h / (p.H / p.groups);
    const int64_t begin = seq_begin(p.seq, n), end = seq_begin(p.seq, n + 1);
    const int slot = p.state_in || p.state_out ? seq_slot(p.seq, n) : -1;

    int r[RL];              // rows past the last one take its inputs and store nothing
    bool live[RL];
    float S[RL][KV][4];
#pragma unroll
    for (int j = 0; j < RL; ++j) {
        const int mine = (slice * RL + j) * 8 + row;
        live[j] = mine < p.P;
        r[j] = live[j] ? mine : p.P - 1;
    }
    auto sat = [&](int j, int k) {
        return (((int64_t)slot * p.H + h) * p.P + r[j]) * p.N + 32 * k + at;
    };
#pragma unroll
    for (int j = 0; j < RL; ++j)
#pragma unroll
        for (int k = 0; k < KV; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                S[j][k][i] = 0.f;
    if (p.state_in && slot >= 0) {
#pragma unroll
        for (int j = 0; j < RL; ++j)
#pragma unroll
            for (int k = 0; k < KV; ++k) {
                if constexpr (WIDE) {
                    if (32 * k + at < p.N) {
                        const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p.state_in + sat(j, k)));
                        S[j][k][0] = v[0], S[j][k][1] = v[1], S[j][k][2] = v[2], S[j][k][3] = v[3];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (32 * k + at + i < p.N)
                            S[j][k][i] = p.state_in[sat(j, k) + i];
                }
            }
    }
    const float a = rate_of_log2(p.a[h]), skip = p.skip ? p.skip[h] : 0.f, bias = p.bias ? p.bias[h] : 0.f;
    const T *xp = static_cast<const T *>(p.x) + begin * p.xst + h * p.xsh;
    const T *dp = static_cast<const T *>(p.dt) + begin * p.dts + h;
    const T *gp = p.gate ? static_cast<const T *>(p.gate) + begin * p.gst + h * p.gsh : nullptr;
    const T *bp = static_cast<const T *>(p.b) + begin * p.bst + group * p.bsg;
    const T *cp = static_cast<const T *>(p.c) + begin * p.cst + group * p.csg;
    T *yp = static_cast<T *>(p.y) + begin * p.yst + h * p.ysh;

    auto load = [&](Token<T, KV, RL> &t) __attribute__((always_inline)) {
        t.dt = *dp;
#pragma unroll
        for (int j = 0; j < RL; ++j) {
            t.x[j] = xp[r[j]];
            if (gp)
                t.gate[j] = gp[r[j]];
        }
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            if constexpr (WIDE) {
                const int n0 = 32 * k + at < p.N ? 32 * k + at : 0;
                __builtin_memcpy(t.b[k], __builtin_assume_aligned(bp + n0, 4 * sizeof(T)), sizeof(t.b[k]));
                __builtin_memcpy(t.c[k], __builtin_assume_aligned(cp + n0, 4 * sizeof(T)), sizeof(t.c[k]));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n0 = 32 * k + at + i < p.N ? 32 * k + at + i : 0;
                    t.b[k][i] = bp[n0];
                    t.c[k][i] = cp[n0];
                }
            }
        }
    };
    auto advance = [&]() __attribute__((always_inline)) {
        xp += p.xst;
        dp += p.dts;
        if (gp)
            gp += p.gst;
        bp += p.bst;
        cp += p.cst;
    };
    auto step = [&](const Token<T, KV, RL> &t) __attribute__((always_inline)) {
        const float d = step_size(load_as_f32(&t.dt) + bias, p.softplus);
        const float decay = __builtin_amdgcn_exp2f(d * a);
#pragma unroll
        for (int j = 0; j < RL; ++j) {
            const float x = load_as_f32(&t.x[j]), dx = d * x;
            float y = 0.f;
#pragma unroll
            for (int k = 0; k < KV; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool in = 32 * k + at + (WIDE ? 0 : i) < p.N;
                    // States past the last one stay zeros, whatever x is.
                    S[j][k][i] = in ? fmaf(decay, S[j][k][i], dx * load_as_f32(&t.b[k][i])) : 0.f;
                    y = in ? fmaf(S[j][k][i], load_as_f32(&t.c[k][i]), y) : y;
                }
            y = lanes_sum<8>(y);
            y = fmaf(skip, x, y);
            if (gp)
                y *= silu(load_as_f32(&t.gate[j]));
            if (live[j] && at == 0)
                store_rne(yp + r[j], y);
        }
        yp += p.yst;
    };
    int64_t left = end - begin;
    if (left > 0) {
        Token<T, KV, RL> t0, t1;
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
        for (int j = 0; j < RL; ++j)
#pragma unroll
            for (int k = 0; k < KV; ++k) {
                if (!live[j])
                    continue;
                if constexpr (WIDE) {
                    if (32 * k + at < p.N)
                        __builtin_nontemporal_store(f32x4{S[j][k][0], S[j][k][1], S[j][k][2], S[j][k][3]},
                                                    reinterpret_cast<f32x4 *>(p.state_out + sat(j, k)));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (32 * k + at + i < p.N)
                            p.state_out[sat(j, k) + i] = S[j][k][i];
                }
            }
    }
}

template <class T, int KV, int RL>
void launch_rows(const HeadScanProblem &p, hipStream_t s)
{
    const int slices = (p.P + 8 * RL - 1) / (8 * RL);
    const int64_t jobs = (int64_t)p.seq.num_seqs * p.H * slices;
    const int waves = jobs <= 1024 ? 1 : 4;     // few waves: one a workgroup, so that they spread over the compute units
    const dim3 grid((unsigned)((jobs + waves - 1) / waves)), block(64 * waves);
    const uintptr_t bc = (uintptr_t)p.b | (uintptr_t)p.c | (uintptr_t)((p.bst | p.bsg | p.cst | p.csg) * (int64_t)sizeof(T));
    const uintptr_t st = (uintptr_t)p.state_in | (uintptr_t)p.state_out;
    if (bc % (4 * sizeof(T)) == 0 && st % 16 == 0 && p.N % 4 == 0)
        hipLaunchKernelGGL((heads_direct_kernel<T, KV, RL, true>), grid, block, 0, s, p, slices);
    else
        hipLaunchKernelGGL((heads_direct_kernel<T, KV, RL, false>), grid, block, 0, s, p, slices);
}

template <class T>
void launch(const HeadScanProblem &p, hipStream_t s)
{
    // Several rows a lane where their states are short and there are rows enough. A token of 16384 rows of 16 states
    // takes 3.5 us with one row a lane and 4.1 with four, of 32768 4.5 and 4.3, of 2^20 64 and 40; of 16384 rows of 64
    // states 4.2 with one and 4.4 with two, of 32768 5.9 and 5.3, of 2^20 99 and 91. Of 128 states one is best: 2^20 rows
    // take 173 us with one and 178 with two.
    const int64_t rows = (int64_t)p.seq.num_seqs * p.H * p.P;
    if (p.N <= 32)
        rows <= 16384 ? launch_rows<T, 1, 1>(p, s) : launch_rows<T, 1, 4>(p, s);
    else if (p.N <= 64)
        rows <= 16384 ? launch_rows<T, 2, 1>(p, s) : launch_rows<T, 2, 2>(p, s);
    else if (p.N <= 128)
        launch_rows<T, 4, 1>(p, s);
    else
        launch_rows<T, 8, 1>(p, s);
}

}  // namespace

// The grid's threads stay below 2^32 (64 a wave of at least 8 rows, up to three waves idle).
bool heads_direct_supports(int num_seqs, int H, int P, int N)
{
    return N <= 256 && (int64_t)num_seqs * H * ((P + 7) / 8) <= (int64_t(1) << 26) - 4;
}

hipError_t launch_heads_direct(const HeadScanProblem &p, hipStream_t s)
{
    if (p.dtype == CONV_BF16)
        launch<uint16_t>(p, s);
    else
        launch<float>(p, s);
    return hipGetLastError();
}

}  // namespace convfwd
