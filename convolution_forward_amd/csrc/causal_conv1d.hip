// Short causal depthwise convolution over packed sequences, channels
// adjacent, with a carried state ("Convolution Is Wx+b Moving Across a
// Signal", section "Where this shows up in models I work with": a causal
// Conv1D pads only before the signal; here the padding is the state).
//
//   y[t,c] = act(bias[c] + sum_j w[c,j] * xx[t - taps + 1 + j, c])
//
// A workgroup takes TT tokens of one sequence (tiles never cross sequences)
// and 512 channels; a thread slides the taps-1 previous rows of its
// channels along the tile in registers, so each row is read once plus taps-1
// rows a tile. The bytes are the time: 8192 tokens of 8192 channels, bf16, 4
// taps, 56 us, 4.8 TB/s (tiles of 32 tokens read 9 % twice; eight rows in
// flight a thread; one at a time took 81 us). 64 sequences of one token: 5.1
// us, the latency of offsets, slot, state and x one after the other. The first
// tile of a sequence also writes the sequence's state, after it has read the
// old one: the two may be the same memory.
#include "common.h"
#include "eight_bit.h"
#include "internal.h"
#include "sequences.h"

namespace convfwd {
namespace {

constexpr int NT = 128;
constexpr int TT = 32;               // tokens of a tile
constexpr int BATCH = 8;             // rows in flight a thread

template <class T, int V>
struct Vec {
    T v[V];
};

template <class T, int V>
__device__ __forceinline__ Vec<T, V> load_raw(const T *p)
{
    Vec<T, V> t;
    if constexpr (V > 1)
        __builtin_memcpy(&t, __builtin_assume_aligned(p, V * sizeof(T)), sizeof(t));
    else
        t.v[0] = *p;
    return t;
}

template <class T, int V>
__device__ __forceinline__ void load_vec(const T *p, float (&f)[V])
{
    const Vec<T, V> t = load_raw<T, V>(p);
#pragma unroll
    for (int i = 0; i < V; ++i)
        f[i] = load_as_f32(&t.v[i]);
}

template <class T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&f)[V])
{
    Vec<T, V> t;
#pragma unroll
    for (int i = 0; i < V; ++i)
        store_rne(&t.v[i], f[i]);
    if constexpr (V > 1) {
        // Streaming stores: 8192 x 8192 bf16 65.2 -> 60.9 us. (Loads keep the
        // caches, where the rows before a tile are found again.)
        typedef uint32_t Piece __attribute__((ext_vector_type(V * sizeof(T) / 4)));
        __builtin_nontemporal_store(__builtin_bit_cast(Piece, t), reinterpret_cast<Piece *>(p));
    } else {
        *p = t.v[0];
    }
}

template <class T, int V, int K>
__global__ __launch_bounds__(NT) void causal_conv1d_kernel(Causal1dProblem p)
{
    const int c = ((int)blockIdx.y * NT + (int)threadIdx.x) * V;
    // The weights' loads go out before the search for the sequence.
    const bool live = c < p.channels;
    T wv[V * K] __attribute__((aligned(V * sizeof(T))));
    float b[V];
    const T *wp = static_cast<const T *>(p.w) + (int64_t)(live ? c : 0) * K;
    if constexpr (V > 1) {
        __builtin_memcpy(wv, __builtin_assume_aligned(wp, V * sizeof(T)), sizeof(wv));     // what the host's rule checks
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i)
            wv[i] = wp[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        b[i] = p.bias ? p.bias[(live ? c : 0) + i] : 0.f;
    const SeqTile tile = seq_tile(p.seq, TT, (int)blockIdx.x);
    if (!live)
        return;
    const int64_t C = p.channels;
    const T *x = static_cast<const T *>(p.x) + tile.begin * p.xs + c;
    T *y = static_cast<T *>(p.y) + tile.begin * p.ys + c;
    const int64_t t0 = (int64_t)tile.index * TT;
    const bool first = tile.index == 0;
    if (t0 >= tile.len && !first)
        return;
    const int slot = p.state_in || p.state_out ? seq_slot(p.seq, tile.n) : -1;
    const T *si = p.state_in && slot >= 0 ? static_cast<const T *>(p.state_in) + (int64_t)slot * (K - 1) * C + c : nullptr;
    // Row t of the sequence; the K-1 before it are the carried ones.
    auto row = [&](int64_t t, float(&f)[V]) {
        if (t >= 0)
            load_vec<T, V>(x + t * p.xs, f);
        else if (si)
            load_vec<T, V>(si + (t + K - 1) * C, f);
        else
#pragma unroll
            for (int i = 0; i < V; ++i)
                f[i] = 0.f;
    };
    float w[K][V], win[K][V];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < K; ++j)
            w[j][i] = load_as_f32(wv + i * K + j);
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
        row(t0 - (K - 1) + j, win[j]);
    const int end = (int)(tile.len - t0 < TT ? tile.len - t0 : TT);
    const T *xt = x + t0 * p.xs;
    T *yt = y + t0 * p.ys;
    auto one = [&](int t) __attribute__((always_inline)) {      // win[K - 1] holds row t
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float a = b[i];
#pragma unroll
            for (int j = 0; j < K; ++j)
                a = fmaf(w[j][i], win[j][i], a);
            // The reciprocal is the instruction's, within 1 ulp; exp's error is |a| 2^-24 of it, that of rounding a.
            f[i] = p.silu ? a * __builtin_amdgcn_rcpf(1.f + __expf(-a)) : a;
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
                win[j][i] = win[j + 1][i];
        }
        store_vec<T, V>(yt + t * p.ys, f);
    };
    int t = 0;
    for (; t + BATCH <= end; t += BATCH) {
        Vec<T, V> rows[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u)
            rows[u] = load_raw<T, V>(xt + (t + u) * p.xs);
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                win[K - 1][i] = load_as_f32(&rows[u].v[i]);
            one(t + u);
        }
    }
    for (; t < end; ++t) {
        load_vec<T, V>(xt + t * p.xs, win[K - 1]);
        one(t);
    }
    if (first && p.state_out && slot >= 0) {
        // Ascending: row r of the new state is row len + r of (old state, x),
        // never an old row that has been overwritten.
        T *so = static_cast<T *>(p.state_out) + (int64_t)slot * (K - 1) * C + c;
#pragma unroll
        for (int r = 0; r < K - 1; ++r) {
            float f[V];
            row(tile.len - (K - 1) + r, f);
            store_vec<T, V>(so + r * C, f);
        }
    }
}

template <class T, int V>
void launch_taps(const Causal1dProblem &p, hipStream_t s)
{
    const int vecs = (p.channels + V - 1) / V;
    const dim3 grid((unsigned)seq_tiles(p.seq, TT), (unsigned)((vecs + NT - 1) / NT));
    switch (p.taps) {
    case 2: hipLaunchKernelGGL((causal_conv1d_kernel<T, V, 2>), grid, dim3(NT), 0, s, p); break;
    case 3: hipLaunchKernelGGL((causal_conv1d_kernel<T, V, 3>), grid, dim3(NT), 0, s, p); break;
    case 4: hipLaunchKernelGGL((causal_conv1d_kernel<T, V, 4>), grid, dim3(NT), 0, s, p); break;
    case 5: hipLaunchKernelGGL((causal_conv1d_kernel<T, V, 5>), grid, dim3(NT), 0, s, p); break;
    case 6: hipLaunchKernelGGL((causal_conv1d_kernel<T, V, 6>), grid, dim3(NT), 0, s, p); break;
    case 7: hipLaunchKernelGGL((causal_conv1d_kernel<T, V, 7>), grid, dim3(NT), 0, s, p); break;
    default: hipLaunchKernelGGL((causal_conv1d_kernel<T, V, 8>), grid, dim3(NT), 0, s, p); break;
    }
}

template <class T>
void launch(const Causal1dProblem &p, hipStream_t s)
{
    // Four channels a thread: with eight bf16 ones the window and the taps took
    // the registers of half the waves (8192 x 8192: 56.9 us against 60.9, 64
    // single tokens 5.1 against 6.3).
    constexpr int V = 4;
    const uintptr_t bits = (uintptr_t)p.x | (uintptr_t)p.y | (uintptr_t)p.w | (uintptr_t)p.state_in | (uintptr_t)p.state_out |
                           (uintptr_t)(p.xs * sizeof(T)) | (uintptr_t)(p.ys * sizeof(T)) |
                           (uintptr_t)(p.channels * sizeof(T));
    if (bits % (V * sizeof(T)) == 0)
        launch_taps<T, V>(p, s);
    else
        launch_taps<T, 1>(p, s);
}

}  // namespace

// Threads of a grid's first axis below 2^32, its second axis within 2^16.
bool causal1d_supports(const Causal1dProblem &p)
{
    return seq_tiles(p.seq, TT) < (int64_t(1) << 24) && p.channels <= (1 << 23);
}

hipError_t launch_causal1d(const Causal1dProblem &p, hipStream_t s)
{
    if (p.dtype == CONV_BF16)
        launch<uint16_t>(p, s);
    else
        launch<float>(p, s);
    return hipGetLastError();
}

}  // namespace convfwd
