// Product of 8-bit operands on the matrix cores: a 1x1 convolution in 8 bits.
//
//   y[m,n] = xs[m] ws[n] sum_k x[m,k] w[n,k] + b[n]
//
// Both operands have K adjacent, so both are staged in LDS as rows of 128
// bytes (a stage is one or two such pieces of K) and a lane's MFMA fragment is 16
// adjacent bytes of a row; the order of K inside a stage is the same for
// both, which is all the sum needs.
//
// Work decomposition: a workgroup takes TM tokens x TN output channels, its
// waves 16*MB x 16*NB pieces of that. Every wave issues its share of a stage's
// loads (straight into LDS, 1 KB a wave instruction: 8 rows of 128 bytes, one
// whole line each) NS - 1 stages ahead, into a ring of NS stages: at the top
// of stage t it waits for its own loads of that stage, and the barrier then
// says both that everyone's have landed and that everyone has read stage
// t - 1, whose place stage t + NS - 1 takes.
//
// w is the MFMA's row operand, so a lane holds four adjacent channels of one
// token. The channel that row 4g + i of block nb stands for is chosen as
// 32 (nb/2) + 8g + 4 (nb%2) + i: two blocks then hold eight adjacent channels
// a lane, and a wave's 16-byte stores fill 64-byte runs of a token's row.
//
// Large products are bound by the matrix instructions and the LDS reads that
// feed them (a wave of the largest tile reads 24 KB for 128x64x128 products):
// int8 8192x8192x4096 in 231 us, 2.38 Pop/s (the library's product without
// scales: 244). e4m3 runs at the bf16 instructions' rate and widens each
// fragment beside them, a third of their time: 8192x8192x4096 in 368-385 us,
// 1.43-1.49 PFLOP/s; 1111x2200x2064 in 20.7 us, 162 tiles on 256 compute units
// and the start and end of them.
#include <type_traits>

#include "common.h"
#include "eight_bit.h"
#include "internal.h"

namespace convfwd {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int KS = 128;                 // K bytes of a piece
constexpr uint32_t OOB = 0x80000000u;
constexpr int BUF_WORD3 = 0x00020000;

template <int N>
__device__ __forceinline__ void wait_vmcnt()
{
    static_assert(N >= 0 && N < 64, "vmcnt holds 6 bits");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <bool E4M3>
struct Acc {
    using type = f32x4;
};
template <>
struct Acc<false> {
    using type = i32x4;
};

// One lane's 16 bytes of an operand as the matrix instructions take them.
// int8: as they are. e4m3: as 16 bf16 values, exactly. The 8-bit float
// instructions keep only some 13 bits of a product's place while they add
// (measured against 64 bits: up to 2^-12.5 of the sum of magnitudes, with
// either instruction), so their sums are not fp32 sums; the bf16 ones add as
// fp32 does.
template <bool E4M3>
struct Frag {
    i32x4 v;
};
template <>
struct Frag<true> {
    bf16x8 v[2];
};

template <bool E4M3>
__device__ __forceinline__ Frag<E4M3> frag(i32x4 raw)
{
    Frag<E4M3> f;
    if constexpr (E4M3) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)raw[i], 1.f, false);
            const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)raw[i], 1.f, true);
            f.v[i >> 1][4 * (i & 1)] = lo[0];
            f.v[i >> 1][4 * (i & 1) + 1] = lo[1];
            f.v[i >> 1][4 * (i & 1) + 2] = hi[0];
            f.v[i >> 1][4 * (i & 1) + 3] = hi[1];
        }
    } else {
        f.v = raw;
    }
    return f;
}

template <bool E4M3>
__device__ __forceinline__ typename Acc<E4M3>::type mma(const Frag<E4M3> &a, const Frag<E4M3> &b, typename Acc<E4M3>::type c)
{
    if constexpr (E4M3) {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[0], b.v[0], c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[1], b.v[1], c, 0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(a.v, b.v, c, 0, 0, 0);
    }
}

// Stored place of 16-byte chunk c of a staged row: the rows of a fragment
// read must fall in distinct 16-byte columns of the 256 bytes that the banks
// span (two rows). x reads 16 adjacent rows; w reads rows 8 (r/4) + r%4 + const.
__device__ __forceinline__ int xswz(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int wswz(int row) { return ((row >> 1) & 1) | (((row >> 3) & 3) << 1); }

struct Q8Args {
    const uint8_t *x, *w;
    const float *xscale, *wscale, *bias;
    void *y;
    int64_t xs, ws, ys;
    int M, N, K;
    int mt, nt;             // tiles
    int group;              // token tiles that one strip of the tile order spans
    int pieces;             // of K
    int stages;             // for the tiles: pieces / SUB, rounded up
    int vec;                // y rows take 16-byte stores
};

// 16 bytes at any address, zeros past the first `left` of them.
__device__ __forceinline__ i32x4 load16_any(const uint8_t *p, int left)
{
    i32x4 v = {0, 0, 0, 0};
    if (left >= 16) {
        __builtin_memcpy(&v, p, 16);
    } else {
#pragma unroll 1
        for (int i = 0; i < left; ++i)
            v[i >> 2] |= (int)((uint32_t)p[i] << (8 * (i & 3)));
    }
    return v;
}

// Where tile number i lies: strips of `group` token tiles, inside a strip
// channel tile by channel tile, so the tiles in flight on an XCD (consecutive
// numbers) share a few rows of each operand in its L2.
__device__ __forceinline__ void place(const Q8Args &a, int i, int &mi, int &ni)
{
    const int strip = i / (a.group * a.nt);
    const int left = a.mt - strip * a.group;
    const int g = left < a.group ? left : a.group;
    const int at = i - strip * a.group * a.nt;
    ni = at / g;
    mi = strip * a.group + at - ni * g;
}

template <int V>
__device__ __forceinline__ void channel_scales(const Q8Args &a, int n, float (&ws)[V], float (&bias)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) {
        ws[i] = n + i < a.N ? a.wscale[n + i] : 0.f;
        bias[i] = n + i < a.N && a.bias ? a.bias[n + i] : 0.f;
    }
}

// V adjacent channels of token m from channel n on: 16-byte stores (8-byte
// ones for four bf16) where y's rows allow them, else one by one.
template <int V, bool OUT_BF16>
__device__ __forceinline__ void store_channels(const Q8Args &a, int m, int n, const float (&v)[V])
{
    using T = std::conditional_t<OUT_BF16, uint16_t, float>;
    T *y = static_cast<T *>(a.y) + (int64_t)m * a.ys + n;
    T o[V] __attribute__((aligned(16)));
#pragma unroll
    for (int i = 0; i < V; ++i)
        if constexpr (OUT_BF16)
            o[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
        else
            o[i] = v[i];
    if (a.vec && n + V <= a.N) {
        typedef uint32_t words __attribute__((ext_vector_type(sizeof(T) * V >= 16 ? 4 : 2)));
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) * V / sizeof(words)); ++i)
            __builtin_nontemporal_store(reinterpret_cast<const words *>(o)[i], reinterpret_cast<words *>(y) + i);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (n + i < a.N)
                y[i] = o[i];
    }
}

template <int MB, int NB, int WM, int WN, int SUB, int NS, bool E4M3, bool OUT_BF16, bool ALIGNED>
__global__ __launch_bounds__(64 * WM * WN) void matmul_q8_kernel(Q8Args a)
{
    using A = typename Acc<E4M3>::type;
    constexpr int TM = 16 * MB * WM, TN = 16 * NB * WN, W = WM * WN;
    constexpr int XB = TM * KS, PIECE = (TM + TN) * KS, STAGE = SUB * PIECE;
    constexpr int LOADS1 = (TM + TN) / 8 / W;       // wave loads of a piece of K: 8 rows each
    constexpr int LOADS = SUB * LOADS1;             // and of a stage
    constexpr int PER = (LOADS1 + 2 * MB - 1) / (2 * MB);
    static_assert(LOADS1 * 8 * W == TM + TN, "whole loads");
    extern __shared__ __align__(16) uint8_t ring[];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 4, r = lane & 15;
    const int bid = with_args_loaded((int)blockIdx.x, a);
    // Workgroup i runs on XCD i % 8: give each XCD consecutive tiles.
    const int tile = (bid & 7) * (int)(gridDim.x >> 3) + (bid >> 3);
    if (tile >= a.mt * a.nt)
        return;
    int mi, ni;
    place(a, tile, mi, ni);
    const int m0 = mi * TM, n0 = ni * TN;

    const uint8_t *xbase = a.x + (int64_t)m0 * a.xs;
    const uint8_t *wbase = a.w + (int64_t)n0 * a.ws;
    const int xrows = min(TM, a.M - m0), wrows = min(TN, a.N - n0);

    // Load v of this wave fills staged rows 8 (W v + wave) .. + 7 (x's TM
    // rows, then w's TN) of each piece; lane L row + L/8, stored chunk L%8.
    static_assert(TM % (8 * W) == 0, "a load belongs to one operand");
    auto row_of = [&](int v) __attribute__((always_inline)) { return 8 * (W * v + wave) + (lane >> 3); };
    auto is_x = [](int v) __attribute__((always_inline)) { return 8 * W * (v + 1) <= TM; };
    auto k_of = [&](int v) __attribute__((always_inline)) {
        const int row = row_of(v);
        return 16 * ((lane & 7) ^ (is_x(v) ? xswz(row) : wswz(row - TM)));
    };

    // Aligned operands go straight into LDS. Rows past the operand and
    // chunks past K read zeros (the range check of the buffer).
    const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(xbase), 0, (int)((xrows - 1) * a.xs + a.K), BUF_WORD3);
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(wbase), 0, (int)((wrows - 1) * a.ws + a.K), BUF_WORD3);
    uint32_t off[ALIGNED ? LOADS1 : 1];
    if constexpr (ALIGNED) {
#pragma unroll
        for (int v = 0; v < LOADS1; ++v) {
            const int row = is_x(v) ? row_of(v) : row_of(v) - TM;
            off[v] = row < (is_x(v) ? xrows : wrows) ? (uint32_t)(row * (int)(is_x(v) ? a.xs : a.ws) + k_of(v)) : OOB;
        }
    }
    // Load v of the piece that starts at k0, into its place at dst.
    auto issue_one = [&](uint8_t *dst, int k0, int v) __attribute__((always_inline)) {
        const uint32_t o = k0 + k_of(v) < a.K ? off[v] + (uint32_t)k0 : OOB;
        const auto to = (__attribute__((address_space(3))) void *)(dst + 1024 * (W * v + wave));
        if (is_x(v))
            __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, to, 16, o, 0, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, to, 16, o, 0, 0, 0);
    };
    // Others go through registers, a stage ahead, and are masked byte by byte at the end of K.
    i32x4 held[ALIGNED ? 1 : LOADS];
    auto fetch = [&](int t) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < LOADS; ++v) {
            const int i = v % LOADS1, row = is_x(i) ? row_of(i) : row_of(i) - TM;
            const int k = (t * SUB + v / LOADS1) * KS + k_of(i);
            held[v] = row < (is_x(i) ? xrows : wrows)
                          ? load16_any((is_x(i) ? xbase : wbase) + row * (is_x(i) ? a.xs : a.ws) + k, a.K - k)
                          : i32x4{0, 0, 0, 0};
        }
    };
    auto put = [&](uint8_t *dst) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < LOADS; ++v)
            *reinterpret_cast<i32x4 *>(dst + v / LOADS1 * PIECE + 1024 * (W * (v % LOADS1) + wave) + 16 * lane) = held[v];
    };

    const int wm = wave / WN, wn = wave % WN;
    // Fragment addresses within a stage.
    int xat[2], wat[NB][2];
    const int xrow = wm * 16 * MB + r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        xat[h] = xrow * KS + 16 * ((4 * h + g) ^ xswz(xrow));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int row = wn * 16 * NB + 32 * (nb >> 1) + 8 * (r >> 2) + 4 * (nb & 1) + (r & 3);
            wat[nb][h] = XB + row * KS + 16 * ((4 * h + g) ^ wswz(row));
        }
    }

    A acc[MB][NB];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            acc[b][nb] = A{0, 0, 0, 0};

    if constexpr (ALIGNED) {
#pragma unroll
        for (int v = 0; v < (NS - 1) * LOADS; ++v)
            issue_one(ring + v / LOADS1 * PIECE, v / LOADS1 * KS, v % LOADS1);
    } else {
        fetch(0);
        put(ring);
    }
    int use = 0, fill = (NS - 1) * STAGE;           // places of stage t and of stage t + NS - 1
    for (int t = 0; t < a.stages; ++t) {
        if constexpr (ALIGNED)
            wait_vmcnt<(NS - 2) * LOADS>();
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!ALIGNED)
            fetch(t + 1);
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub) {
            const uint8_t *s = ring + use + sub * PIECE;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                Frag<E4M3> wf[NB];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    wf[nb] = frag<E4M3>(*reinterpret_cast<const i32x4 *>(s + wat[nb][h]));
#pragma unroll
                for (int b = 0; b < MB; ++b) {
                    const Frag<E4M3> xf = frag<E4M3>(*reinterpret_cast<const i32x4 *>(s + xat[h] + b * 16 * KS));
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                        acc[b][nb] = mma<E4M3>(wf[nb], xf, acc[b][nb]);
                    if constexpr (ALIGNED) {
                        // The next loads, a few between the products: a wave is held some 150 clocks for each of
                        // them, and all at once they left the matrix cores idle (265 us against 243 at
                        // 8192x8192x4096). Products and loads keep their order; LDS reads and VALU work may move
                        // across.
                        __builtin_amdgcn_sched_barrier(0x386);
#pragma unroll
                        for (int v = (h * MB + b) * PER; v < (h * MB + b + 1) * PER; ++v)
                            if (v < LOADS1)
                                issue_one(ring + fill + sub * PIECE, ((t + NS - 1) * SUB + sub) * KS, v);
                    }
                }
            }
        }
        if constexpr (!ALIGNED)
            put(ring + fill);
        use = use + STAGE == NS * STAGE ? 0 : use + STAGE;
        fill = fill + STAGE == NS * STAGE ? 0 : fill + STAGE;
    }
    // The stages past the end (zeros) land before the workgroup's LDS is let go.
    wait_vmcnt<0>();

    // Lane (g, r) holds, of token 16 b + r of the wave's, channels 32 p + 8 g .. + 7 in blocks 2p and 2p + 1.
    const int nw = n0 + wn * 16 * NB + 8 * g;
    float ws[NB / 2][8], bias[NB / 2][8];
#pragma unroll
    for (int p = 0; p < NB / 2; ++p)
        channel_scales<8>(a, nw + 32 * p, ws[p], bias[p]);
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int m = m0 + wm * 16 * MB + 16 * b + r;
        if (m >= a.M)
            continue;
        const float xsc = a.xscale[m];
#pragma unroll
        for (int p = 0; p < NB / 2; ++p) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = (float)acc[b][2 * p + (i >> 2)][i & 3] * xsc * ws[p][i] + bias[p][i];
            store_channels<8, OUT_BF16>(a, m, nw + 32 * p, v);
        }
    }
}

// Few tokens (at most 16 MB a workgroup): w's bytes are the time, so w goes
// straight from memory into MFMA fragments, and K is split over the
// workgroup's eight waves to have as many loads in flight as there is w.
// (8 x 4096 x 4096 int8: 6.0-6.5 us with w in memory, 2.7 TB/s, 5.4 with it in
// the caches; 2 us of it are the launch and the first load's latency.)
// Wave i takes K pieces i, i + 8, ... of 128 bytes, four at a time, and the
// eight partial sums of a 16-channel block meet in LDS (in a fixed order).
constexpr int SW = 8;

template <int MB, bool E4M3, bool OUT_BF16, bool ALIGNED>
__global__ __launch_bounds__(64 * SW) void matmul_q8_few_kernel(Q8Args a)
{
    using A = typename Acc<E4M3>::type;
    __shared__ A part[SW][MB][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 4, r = lane & 15;
    const int n0 = with_args_loaded((int)blockIdx.x, a) * 16;
    const int m0 = (int)blockIdx.y * 16 * MB;
    // Rows past the operand read its last row; their outputs are not stored.
    const uint8_t *wrow = a.w + (int64_t)min(n0 + r, a.N - 1) * a.ws + 16 * g;
    const uint8_t *xrow[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b)
        xrow[b] = a.x + (int64_t)min(m0 + 16 * b + r, a.M - 1) * a.xs + 16 * g;
    A acc[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b)
        acc[b] = A{0, 0, 0, 0};
    auto load = [&](const uint8_t *row, int k) __attribute__((always_inline)) {
        if constexpr (ALIGNED)
            return k + 16 * g < a.K ? *reinterpret_cast<const i32x4 *>(row + k) : i32x4{0, 0, 0, 0};
        else
            return load16_any(row + k, a.K - k - 16 * g);
    };
    constexpr int U = 4;
    for (int t = wave; t < a.pieces; t += SW * U) {
        i32x4 wf[U][2], xf[U][MB][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (t + SW * u) * KS + 64 * h;
                wf[u][h] = load(wrow, k);
#pragma unroll
                for (int b = 0; b < MB; ++b)
                    xf[u][b][h] = load(xrow[b], k);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const Frag<E4M3> w = frag<E4M3>(wf[u][h]);
#pragma unroll
                for (int b = 0; b < MB; ++b)
                    acc[b] = mma<E4M3>(w, frag<E4M3>(xf[u][b][h]), acc[b]);
            }
    }
#pragma unroll
    for (int b = 0; b < MB; ++b)
        part[wave][b][lane] = acc[b];
    __syncthreads();
    // Wave b joins token block b; lane (g, r) has channels 4g .. 4g + 3 of token r.
    if (wave >= MB)
        return;
    A sum = part[0][wave][lane];
#pragma unroll
    for (int i = 1; i < SW; ++i)
        sum += part[i][wave][lane];
    const int m = m0 + 16 * wave + r, n = n0 + 4 * g;
    if (m >= a.M)
        return;
    float ws[4], bias[4], v[4];
    channel_scales<4>(a, n, ws, bias);
    const float xsc = a.xscale[m];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = (float)sum[i] * xsc * ws[i] + bias[i];
    store_channels<4, OUT_BF16>(a, m, n, v);
}

template <int MB, int NB, int WM, int WN, int SUB, int NS, bool E4M3, bool OB, bool ALIGNED>
hipError_t launch_tiles(Q8Args &a, hipStream_t s)
{
    constexpr int TM = 16 * MB * WM, TN = 16 * NB * WN;
    constexpr int lds = NS * SUB * (TM + TN) * KS;
    static_assert(lds <= 160 * 1024, "LDS");
    a.mt = (a.M + TM - 1) / TM;
    a.nt = (a.N + TN - 1) / TN;
    a.group = 8;
    a.stages = (a.pieces + SUB - 1) / SUB;
    const int64_t tiles = (int64_t)a.mt * a.nt;
    const hipError_t attr = allow_lds<matmul_q8_kernel<MB, NB, WM, WN, SUB, NS, E4M3, OB, ALIGNED>>(lds);
    if (attr != hipSuccess)
        return attr;
    hipLaunchKernelGGL((matmul_q8_kernel<MB, NB, WM, WN, SUB, NS, E4M3, OB, ALIGNED>), dim3((unsigned)((tiles + 7) / 8 * 8)),
                       dim3(64 * WM * WN), lds, s, a);
    return hipGetLastError();
}

// Tiles, and whether a grid of them (whole eights of workgroups) stays below 2^32 threads.
int64_t tiles_of(int64_t M, int N, int tm, int tn) { return ((M + tm - 1) / tm) * (((int64_t)N + tn - 1) / tn); }
bool fits(int64_t workgroups, int threads) { return (workgroups + 7) / 8 * 8 * threads < (int64_t(1) << 32); }

template <int MB, bool E4M3, bool OB, bool ALIGNED>
hipError_t launch_few(const Q8Args &a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)((a.M + 16 * MB - 1) / (16 * MB)));
    hipLaunchKernelGGL((matmul_q8_few_kernel<MB, E4M3, OB, ALIGNED>), grid, dim3(64 * SW), 0, s, a);
    return hipGetLastError();
}

template <bool E4M3, bool OB, bool ALIGNED>
hipError_t launch(Q8Args &a, hipStream_t s)
{
    // Up to 32 tokens the few-token form is the faster one (8 x 4096 x 4096:
    // 6.5 us against 9.4 on 64x64 tiles; 32: 9.0 against 9.7), past that the
    // tiles are (64 x 8192 x 4096: 13.9 us against 24).
    const bool few = fits(((int64_t)a.N + 15) / 16, 64 * SW);
    if (a.M <= 16 && few)
        return launch_few<1, E4M3, OB, ALIGNED>(a, s);
    if (a.M <= 32 && few)
        return launch_few<2, E4M3, OB, ALIGNED>(a, s);
    // The tile whose rounds over the 256 compute units cost least. A round's
    // cost is its time at K = 4096 over the 64x64 tile's (int8, from 32x64 up:
    // 8.5, 8.9, 12.5, 17.3, 27, 43 us; e4m3 13.3, 15.8, 20, 32, 49, 81): the larger a tile, the fewer
    // bytes it loads for each product, and the longer it holds its unit. (1024
    // x 8192 x 4096: 128x256 36 us, 128x128 45, 256x256 52; 512 x 4096 x
    // 4096: 64x128 14.7, 64x64 17.7, 128x128 19; 64 x 8192 x 4096: 32x64 11.0,
    // 64x64 12.5, in e4m3 13.9 and 16.1; 256 x 4096 x 4096: 64x64 9.2, 32x64 11.4.)
    auto cost = [&](int tm, int tn, int each) {
        const int64_t tiles = tiles_of(a.M, a.N, tm, tn);
        return fits(tiles, 512) ? (tiles + 255) / 256 * each : INT64_MAX;
    };
    const int64_t costs[6] = {cost(256, 256, 48), cost(128, 256, 31), cost(128, 128, 20), cost(64, 128, 14),
                              cost(64, 64, 10), cost(32, 64, 9)};
    int best = 0;
    for (int i = 1; i < 6; ++i)
        if (costs[i] < costs[best])
            best = i;
    switch (best) {
    case 0: return launch_tiles<8, 4, 2, 4, 1, 2, E4M3, OB, ALIGNED>(a, s);
    case 1: return launch_tiles<4, 4, 2, 4, 1, ALIGNED ? 3 : 2, E4M3, OB, ALIGNED>(a, s);
    case 2: return launch_tiles<4, 2, 2, 4, 1, ALIGNED ? 3 : 2, E4M3, OB, ALIGNED>(a, s);
    case 3: return launch_tiles<2, 2, 2, 4, 1, ALIGNED ? 3 : 2, E4M3, OB, ALIGNED>(a, s);
    case 4: return launch_tiles<1, 2, 4, 2, 2, ALIGNED ? 3 : 2, E4M3, OB, ALIGNED>(a, s);
    default: return launch_tiles<1, 2, 2, 2, 2, ALIGNED ? 3 : 2, E4M3, OB, ALIGNED>(a, s);
    }
}

}  // namespace

// Every stride must let a tile's byte offsets stay below 2^31, and the largest tiles must fit a grid.
bool matmul_q8_tiled_supports(const MatmulQ8Problem &p)
{
    return p.xs <= (1 << 22) && p.ws <= (1 << 22) && fits(tiles_of(p.M, p.N, 256, 256), 512);
}

hipError_t launch_matmul_q8(const MatmulQ8Problem &p, hipStream_t s)
{
    Q8Args a = {};
    a.x = static_cast<const uint8_t *>(p.x);
    a.w = static_cast<const uint8_t *>(p.w);
    a.xscale = p.xscale;
    a.wscale = p.wscale;
    a.bias = p.bias;
    a.y = p.y;
    a.xs = p.xs;
    a.ws = p.ws;
    a.ys = p.ys;
    a.M = (int)p.M;
    a.N = p.N;
    a.K = p.K;
    a.pieces = (p.K + KS - 1) / KS;
    const bool bf = p.ydt == CONV_BF16, e = p.qdt == CONV_E4M3;
    a.vec = ((uintptr_t)p.y | (uintptr_t)(p.ys * (bf ? 2 : 4))) % 16 == 0;
    const bool aligned =
        (((uintptr_t)p.x | (uintptr_t)p.w | (uintptr_t)p.xs | (uintptr_t)p.ws | (uintptr_t)p.K) & 15) == 0;
    if (aligned)
        return e ? (bf ? launch<true, true, true>(a, s) : launch<true, false, true>(a, s))
                 : (bf ? launch<false, true, true>(a, s) : launch<false, false, true>(a, s));
    return e ? (bf ? launch<true, true, false>(a, s) : launch<true, false, false>(a, s))
             : (bf ? launch<false, true, false>(a, s) : launch<false, false, false>(a, s));
}

}  // namespace convfwd
