// The selective scan with one decay a head, by chunks of 64 tokens on the
// matrix cores, bf16 or fp32 operands, in fp32 precision.
//
// Inside a chunk let L_i be the sum of the exponents d a up to token i and S
// [P,N] the state before the chunk. The 64 steps are
//   Y  = diag(exp L) C S^T + M X,   M_ij = exp(L_i - L_j) d_j (c_i . b_j) for j <= i, else 0
//   S' = exp(L_63) S + X^T diag(d_j exp(L_63 - L_j)) B
// with the skipped input on M's diagonal. Sums and differences of L are taken
// in 64 bits, so a strong decay early in a chunk costs the later ones nothing.
//
// A wave owns 16 rows of S (columns of X) of one head and keeps them in its
// accumulators from chunk to chunk; as they leave one product they are the
// operand of the next. The waves of a workgroup (eight in bf16, four in fp32)
// are of one group and share the chunk's B and C in LDS. M's six blocks of 16 x
// 32 go round the waves of its head, which make c . b and the factors for them,
// each head's anew.
//
// Long sequences are cut into segments of `seg` tokens where there are too few
// heads to fill the chip: a first kernel makes the state that each segment but
// a sequence's last leaves of nothing (the first one's: of the sequence's own
// state), the last one goes over all segments and puts together the state before
// each from those of the segments before it. Where these may be more than
// FOLDED a kernel between the two has done that.
//
// Precision: bf16 operands (B, C, X) are exact; every other operand (S, M, X
// with its factors) and each fp32 one is split into three bf16 parts, x = hi +
// mid + lo, 24 bits together, and the products of parts are added in fp32: three
// for an exact operand times a split one, eight for two split ones. (Parts are
// cut, so mid may be 2^-7 of x and lo 2^-15; lo lo is left out, 2^-30. Without
// mid lo and lo mid, 2^-21 together, 8192 tokens of 128 heads in fp32 take 919 us
// instead of 966; parts rounded to nearest, whose mid lo is 2^-25, 953, but hi
// hi may then leave fp32's range where the product does not.)
//
// 8192 tokens of 128 heads of 64 x 128 in 8 groups, bf16: 264 to 281 us, 1.65
// TB/s, a quarter of it the first kernel. The matrix instructions of both,
// counting the products of parts, are 133 us at a large product's rate. By the
// counters they run in 25 % of the first kernel's clocks and 28 % of the last
// one's, vector instructions (splits, factors, gates) are issued in 46 and 58
// %, and LDS is busy in 28 and 37 %; what keeps these from overlapping more is
// that a chunk's phases follow each other, two barriers in the first kernel and
// three in the last, with 2.6 and 3 waves a SIMD.
//
// Values that are not finite: a zero of M times a NaN would carry it to earlier
// tokens. So values of X, B and the step sizes that are not finite are read as
// zeros and their token is noted; outputs from it on, and the state, are set to
// NaN: a row of a head (X), a head (the step size or the exponent) or a group (B).
#include <type_traits>

#include "common.h"
#include "eight_bit.h"
#include "internal.h"
#include "scan_math.h"
#include "sequences.h"

namespace convfwd {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr int Q = 64;                   // tokens of a chunk
constexpr int NT_JOIN = 64;
// Segments of a sequence whose states the last kernel puts together by itself. Whole calls: 6 sequences of 4095 tokens
// together, 16 segments, 95 us, with a kernel of its own for that 112; 8192 tokens of 128 heads, 8 segments, 264 and 275;
// 16384 tokens of 32 heads, 64 segments, 129 and 122.
constexpr int FOLDED = 16;
constexpr int NEVER = 0x7fffffff;
constexpr int FRAG = 1024;              // 64 lanes x 16 bytes
constexpr int MFRAGS = 6;               // 16 x 32 blocks of a lower triangle of 64

struct HeadsArgs {
    HeadScanProblem p;
    float *states;          // workspace: a state for each segment number ...
    float *decays;          // ... and its decay for each head
    int seg;                // tokens of a segment
    int units;              // segment numbers x groups
    int slices;             // slices of 16 columns a head
    int jobs;               // slices that a workgroup takes (waves past them help with what is shared)
    int wgs;                // workgroups of a segment and group
    int heads;              // most heads a workgroup's jobs belong to
    bool joined;            // the state before each segment is there, not what each one leaves
};

// What a chunk's exponents come to for one head: what M needs, and what the
// products after it do, while the next chunk's are made.
struct __align__(16) Factors {
    double L[Q];            // in units of log 2
    float step[Q];          // d
    float row[Q];           // 2^(L - L_31)
    float col[Q];           // 2^(L_31 - L) d
    struct __align__(16) {
        float up[Q];        // 2^L
        float tail[Q];      // 2^(L_63 - L) d
        float total;        // 2^L_63
        int wide;           // row and col may leave fp32's range
        int bad;            // first token whose step is not finite, or its exponent no number
    } of[2];
};

// A barrier for LDS traffic only: __syncthreads would also wait for the loads
// of the next chunk that are in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Eight values as three bf16 parts each, every part what the ones before left,
// cut to bf16's eight bits: together exactly the value (down to fp32's smallest
// normal number times 2^16). Masks and subtractions, 2.7 clocks a wave beside
// others; rounding conversions and shifts would take 4.4. (A remainder is one
// v_dot2_f32_bf16 too, but those share the matrix cores: beside a wave of matrix
// instructions one takes 22 clocks.)
__device__ __forceinline__ void split8(const float (&x)[8], bf16x8 (&part)[3])
{
    u32x4 packed[3];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        float a = x[2 * h], b = x[2 * h + 1];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            packed[i][h] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
            if (i < 2) {
                a -= __uint_as_float(__float_as_uint(a) & 0xffff0000u);
                b -= __uint_as_float(__float_as_uint(b) & 0xffff0000u);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
        part[i] = __builtin_bit_cast(bf16x8, packed[i]);
}

// acc += a b, each of one exact part or three: small products first.
template <int NA, int NB>
__device__ __forceinline__ f32x4 product(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], f32x4 acc)
{
#pragma unroll
    for (int k = NA + NB > 4 ? 3 : 2; k >= 0; --k)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (k - i >= 0 && k - i < NB)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[k - i], acc, 0, 0, 0);
    return acc;
}

// Four values of a column: of each 16 lanes, lane i gets value i % 4 of the
// places of lanes i / 4, 4 + i / 4, 8 + i / 4 and 12 + i / 4.
__device__ __forceinline__ bf16x4 transposed(const void *place)
{
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                          (__attribute__((address_space(3))) i16x4 *)(place)));
}

__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// A double from another lane (a DPP control), or zero: lanes shifted from
// outside their row of 16, and rows that ROWS leaves out.
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0u, (uint32_t)u, CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0u, (uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double of_lane(double v, int lane)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, lane), hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// 2^x to an ulp or two whatever x is (the instruction's error grows with |x| only through its argument's rounding).
__device__ __forceinline__ float power2(double x)
{
    const double n = rint(x);
    return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f((float)(x - n)), (int)n);
}

// Whether any of a piece's values is infinite or NaN: an exponent of all ones carries into the bit above it.
template <bool F32>
__device__ __forceinline__ uint32_t not_finite(const u32x4 &v)
{
    constexpr uint32_t E = F32 ? 0x7f800000u : 0x7f807f80u, ONE = F32 ? 0x00800000u : 0x00800080u;
    return (((v[0] & E) + ONE) | ((v[1] & E) + ONE) | ((v[2] & E) + ONE) | ((v[3] & E) + ONE)) & ~(E | (ONE - 1)) &
           (F32 ? 0x80000000u : 0x80008000u);
}

// KN steps of 32 states (N up to 32 KN), CW columns a wave.
// FULL: outputs and final states; else the states that segments leave. VEC:
// 16-byte pieces of x, b, c and gate, and of states (a host rule).
template <class T, int KN, int WAVES, bool FULL, bool VEC>
struct Chunks {
    static constexpr int NT = 64 * WAVES;
    static constexpr bool F32 = std::is_same<T, float>::value;
    static constexpr int XP = F32 ? 3 : 1;          // parts of an operand as it lies in memory
    static constexpr int E = 16 / sizeof(T);        // values of a piece
    static constexpr int NP = 32 * KN, RC = 4 * KN; // states of a row in LDS, in pieces of eight
    static constexpr int PB = Q * NP / E / NT;      // pieces of B, and of C, a thread
    static constexpr int CW = 16;                   // columns of a wave
    static constexpr int PX = Q * CW / E / 64;      // pieces of X a lane
    // LDS: B, C (each XP parts), then X of each wave (XP parts) which M takes the place of, then the factors and notes.
    // Rows of C are a piece longer than their states, so that 16 of them begin in 16 different groups of four banks;
    // those of B four pieces, and each eight of them another, which keeps apart both the rows 8 i + j (i, j < 4) of a
    // fragment and the four pieces of four rows of a transposed read. (Pieces exchanged within a row would do so
    // without the room, but then every place is an address of its own, and they took 50 registers.)
    static constexpr int BROW = (RC + 4) * 16, CROW = (RC + 1) * 16;
    static constexpr int BBYTES = Q * BROW + Q / 8 * 16, CBYTES = Q * CROW, XBYTES = Q * CW * 2;
    static constexpr int C_AT = XP * BBYTES, X_AT = C_AT + (FULL ? XP * CBYTES : 0);

    static __host__ __device__ int shared_at(int heads)
    {
        const int x = WAVES * XP * XBYTES, m = FULL ? heads * MFRAGS * 3 * FRAG : 0;
        return X_AT + (x > m ? x : m);
    }
    static __host__ __device__ int lds(int heads)
    {
        return shared_at(heads) + heads * (int)sizeof(Factors) + WAVES * CW * 4 + 16;
    }

    static __host__ __device__ constexpr int b_place(int row, int piece) { return row * BROW + (row >> 3) * 16 + piece * 16; }
    static __host__ __device__ constexpr int c_place(int row, int piece) { return row * CROW + piece * 16; }

    static __device__ __forceinline__ void run(const HeadsArgs &a)
    {
        const HeadScanProblem &p = a.p;
        extern __shared__ __align__(16) uint8_t lds_[];
        uint8_t *const bs = lds_, *const cs = lds_ + C_AT, *const xm = lds_ + X_AT;
        uint8_t *const after = lds_ + shared_at(a.heads);
        Factors *const factors = reinterpret_cast<Factors *>(after);                    // [heads]
        int *const badcol = reinterpret_cast<int *>(after + a.heads * sizeof(Factors));
        int *const badb = badcol + WAVES * CW;                                          // [2]

        // Workgroup i runs on XCD i % 8: those of one segment and group, which
        // read the same B and C, go to one XCD and meet in its L2.
        const int at = (int)blockIdx.x >> 3;
        const int wg = at % a.wgs, unit = at / a.wgs * 8 + ((int)blockIdx.x & 7);
        if (unit >= a.units)
            return;
        const int group = unit % p.groups, number = unit / p.groups;
        const SeqTile tile = seq_tile(p.seq, a.seg, number);
        // (The same in all lanes, which the compiler has to be told: descriptors follow from it.)
        const int index = __builtin_amdgcn_readfirstlane(tile.index);
        const int whole = __builtin_amdgcn_readfirstlane((int)tile.len);
        const int64_t t0 = (int64_t)index * a.seg;
        if (t0 >= whole && index != 0)
            return;
        const bool last = t0 + a.seg >= whole;
        if (!FULL && last)
            return;
        const int64_t first = __builtin_amdgcn_readfirstlane((int)tile.begin) + t0;
        const int len = last ? whole - (int)t0 : a.seg;
        const int chunks = (len + Q - 1) / Q;

        int tid = threadIdx.x, lane = tid & 63;
        int w = __builtin_amdgcn_readfirstlane(tid >> 6);
        int g = lane >> 4, c = lane & 15;
        const int per = p.H / p.groups, group_jobs = per * a.slices;
        const int job0 = wg * a.jobs, job1 = min(job0 + a.jobs, group_jobs);
        const int head0 = job0 / a.slices, heads = (job1 - 1) / a.slices - head0 + 1;    // of this workgroup, in the group
        const bool mine = job0 + w < job1;          // whether this wave has columns
        const int job = mine ? job0 + w : job0;
        const int hi = job / a.slices - head0;      // its head, of the workgroup's
        const int h = group * per + head0 + hi;
        const int col0 = job % a.slices * CW;

        // ---- Loads.
        // VEC: through buffer descriptors of a chunk's rows that there are, whose
        // end turns loads past it into zeros and drops stores (a host rule keeps
        // a chunk within 2^31 bytes and rows from overlapping). A lane's offset
        // of a column that is not there is past any end.
        constexpr uint32_t NOWHERE = 0x80000000u;
        auto view = [&](const T *base, int64_t stride, int rows, int width) __attribute__((always_inline)) {
            const int end = rows > 0 ? (rows - 1) * (int)stride + width : 0;
            return __builtin_amdgcn_make_buffer_rsrc(const_cast<T *>(base), 0, (uint32_t)(end * (int)sizeof(T)), 0x00020000);
        };
        auto offset_of = [&](int row, int col, int64_t stride, int width) __attribute__((always_inline)) {
            return col < width ? (uint32_t)((row * (int)stride + col) * (int)sizeof(T)) : NOWHERE;
        };
        const T *xp = static_cast<const T *>(p.x) + first * p.xst + h * p.xsh + col0;
        const T *gp = p.gate ? static_cast<const T *>(p.gate) + first * p.gst + h * p.gsh + col0 : xp;
        const int64_t gst = p.gate ? p.gst : p.xst;
        const T *bp = static_cast<const T *>(p.b) + first * p.bst + group * p.bsg;
        const T *cp = static_cast<const T *>(p.c) + first * p.cst + group * p.csg;
        T *yp = static_cast<T *>(p.y) + first * p.yst + h * p.ysh + col0;
        // Wave w < heads makes the factors of head head0 + w.
        const int fh = group * per + head0 + min(w, heads - 1);
        const T *dp = static_cast<const T *>(p.dt) + first * p.dts + fh;
        const double rate = (double)(p.a[fh] < -FLT_MAX ? -FLT_MAX : p.a[fh]) * 1.4426950408889634074;   // as rate_of_log2
        const float bias = p.bias ? p.bias[fh] : 0.f;
        const int cols = p.P - col0;                // columns there are, from the wave's first

        // The gate (x in its place where there is none) of the columns V g + .. of tokens 16 it + c.
        constexpr int V = 4;
        struct Gate {
            T v[V] __attribute__((aligned(V * sizeof(T))));
        };
        u32x4 bv[PB], cv[FULL ? PB : 1], xv[PX];
        Gate gate[FULL ? 4 : 1];
        T dv;
        uint32_t xo = offset_of(lane / (CW / E), lane % (CW / E) * E, p.xst, cols);
        uint32_t bo = offset_of(tid / (NP / E), tid % (NP / E) * E, p.bst, p.N);
        uint32_t co = offset_of(tid / (NP / E), tid % (NP / E) * E, p.cst, p.N);
        uint32_t go = offset_of(c, V * g, gst, cols);
        // A piece of a row; the values that are not there are zeros.
        auto piece = [&](const T *row, int col, int width) __attribute__((always_inline)) {
            T v[E] __attribute__((aligned(16))) = {};
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (col + e < width)
                    v[e] = row[col + e];
            return *reinterpret_cast<const u32x4 *>(v);
        };
        // What a chunk loads: pieces of X, B, C and the gate, in this order. One at a time: a load holds its wave some
        // 150 clocks, which the products before it fill. Chunks past the last one load nothing.
        constexpr int LOADS = PX + PB + (FULL ? PB + 4 : 0);
        auto load = [&](int ch, int k) __attribute__((always_inline)) {
            const int rows = min(len - ch * Q, Q);
            const int64_t at0 = (int64_t)ch * Q;
            if (k < PX) {
                const T *base = xp + at0 * p.xst;
                const int row = (k * 64 + lane) / (CW / E), col = (k * 64 + lane) % (CW / E) * E;
                if constexpr (VEC)
                    xv[k] = __builtin_amdgcn_raw_buffer_load_b128(view(base, p.xst, rows, cols),
                                                                  xo + k * (64 * E / CW * (int)sizeof(T)) * (int)p.xst, 0, 0);
                else if (rows > 0)
                    xv[k] = piece(base + min(row, rows - 1) * p.xst, col, cols);
            } else if (k < PX + (FULL ? 2 : 1) * PB) {
                const int i = (k - PX) % PB;
                const bool of_b = k < PX + PB;
                const int64_t st = of_b ? p.bst : p.cst;
                const T *base = (of_b ? bp : cp) + at0 * st;
                const int row = (i * NT + tid) / (NP / E), col = (i * NT + tid) % (NP / E) * E;
                u32x4 &to = of_b ? bv[i] : cv[FULL ? i : 0];
                if constexpr (VEC)
                    to = __builtin_amdgcn_raw_buffer_load_b128(
                        view(base, st, rows, p.N), (of_b ? bo : co) + i * (NT * E / NP * (int)sizeof(T)) * (int)st, 0, 0);
                else if (rows > 0)
                    to = piece(base + min(row, rows - 1) * st, col, p.N);
            } else {
                const int it = k - PX - 2 * PB;
                const T *base = gp + at0 * gst;
                if constexpr (VEC) {
                    const auto r = view(base, gst, rows, cols);
                    const uint32_t o = go + it * (16 * (int)sizeof(T)) * (int)gst;
                    if constexpr (sizeof(Gate) == 16)
                        gate[it] = __builtin_bit_cast(Gate, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0));
                    else
                        gate[it] = __builtin_bit_cast(Gate, __builtin_amdgcn_raw_buffer_load_b64(r, o, 0, 0));
                } else if (rows > 0) {
                    const T *gr = base + min(16 * it + c, rows - 1) * gst;
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        gate[it].v[e] = gr[V * g + e < cols ? V * g + e : 0];
                }
            }
        };
        auto load_step = [&](int ch) __attribute__((always_inline)) {
            const int64_t t = min(ch * Q + lane, len - 1);
            dv = dp[t * p.dts];
        };
        // A piece's parts into LDS: in bf16 the piece itself, in fp32 half a piece of each part (cut as in split8;
        // rounded, values next to fp32's largest would leave bf16's range).
        auto put = [&](uint8_t *at16, int part_bytes, const u32x4 &v, int half) __attribute__((always_inline)) {
            if constexpr (F32) {
                f32x4 left = __builtin_bit_cast(f32x4, v);
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    u32x2 t;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        t[e] = __builtin_amdgcn_perm(__float_as_uint(left[2 * e + 1]), __float_as_uint(left[2 * e]), 0x07060302u);
                    *reinterpret_cast<u32x2 *>(at16 + i * part_bytes + 8 * half) = t;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        left[e] -= __uint_as_float(__float_as_uint(left[e]) & 0xffff0000u);
                }
            } else {
                *reinterpret_cast<u32x4 *>(at16) = v;
            }
        };
        // Values that are not finite -> zeros, and note(their column).
        auto look = [&](u32x4 &v, auto note) __attribute__((always_inline)) {
            T e[E] __attribute__((aligned(16)));
            *reinterpret_cast<u32x4 *>(e) = v;
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (!(fabsf(load_as_f32(&e[i])) < INFINITY)) {
                    note(i);
                    e[i] = T(0);
                }
            v = *reinterpret_cast<const u32x4 *>(e);
        };
        auto put_bc = [&](int ch) __attribute__((always_inline)) {
            const int rows = min(len - ch * Q, Q);
            uint32_t odd = 0;
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                if (!VEC && (i * NT + tid) / (NP / E) >= rows)
                    bv[i] = u32x4{0, 0, 0, 0};
                odd |= not_finite<F32>(bv[i]);
            }
            if (__any(odd != 0)) {
#pragma unroll
                for (int i = 0; i < PB; ++i)
                    look(bv[i], [&](int) { atomicMin(badb + (ch & 1), (i * NT + tid) / (NP / E)); });
            }
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                const int row = (i * NT + tid) / (NP / E), col = (i * NT + tid) % (NP / E) * E;
                put(bs + b_place(row, col / 8), BBYTES, bv[i], col / 4 & 1);
                if constexpr (FULL)
                    put(cs + c_place(row, col / 8), CBYTES, cv[i], col / 4 & 1);
            }
        };
        // X of the wave's columns through its own part of LDS, as 8 tokens of a column a lane.
        bf16x8 xf[2][XP];
        auto put_x = [&](int ch) __attribute__((always_inline)) {
            const int rows = min(len - ch * Q, Q);
            uint8_t *const own = xm + w * XP * XBYTES;
            uint32_t odd = 0;
#pragma unroll
            for (int i = 0; i < PX; ++i) {
                if (!VEC && (i * 64 + lane) / (CW / E) >= rows)
                    xv[i] = u32x4{0, 0, 0, 0};
                odd |= not_finite<F32>(xv[i]);
            }
            if (__any(odd != 0)) {
#pragma unroll
                for (int i = 0; i < PX; ++i) {
                    const int row = (i * 64 + lane) / (CW / E), col = (i * 64 + lane) % (CW / E) * E;
                    look(xv[i], [&](int e) { atomicMin(badcol + w * CW + col + e, row); });
                }
            }
#pragma unroll
            for (int i = 0; i < PX; ++i) {
                const int row = (i * 64 + lane) / (CW / E), col = (i * 64 + lane) % (CW / E) * E;
                put(own + row * CW * 2 + col / 8 * 16, XBYTES, xv[i], col / 4 & 1);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < XP; ++i) {
                    const uint8_t *t = own + i * XBYTES + (32 * s + 8 * g + (c >> 2)) * CW * 2 + (c & 3) * 8;
                    xf[s][i] = join(transposed(t), transposed(t + 4 * CW * 2));
                }
        };
        double exponent = 0.0;      // of the whole segment, in wave w < heads
        auto make_factors = [&](int ch) __attribute__((always_inline)) {
            if (w >= heads)
                return;
            Factors &f = factors[w];
            auto &of = f.of[ch & 1];
            float d = step_size(load_as_f32(&dv) + bias, p.softplus);
            // Exponents past +-10000 are 0 and infinity either way.
            double e = (double)d * rate;
            const bool here = lane < len - ch * Q;
            const bool bad = here && (!(fabsf(d) < INFINITY) || e != e);
            e = fmin(fmax(e, -1e4), 1e4);
            const uint64_t bads = __ballot(bad);
            if (!here || bad) {
                d = 0.f;
                e = 0.0;
            }
            // Sums up to each lane: within 16 lanes, then of the rows of 16 before.
            e += moved<0x111, 0xf>(e);
            e += moved<0x112, 0xf>(e);
            e += moved<0x114, 0xf>(e);
            e += moved<0x118, 0xf>(e);
            e += moved<0x142, 0xa>(e);
            e += moved<0x143, 0xc>(e);
            const double mid = of_lane(e, 31), end = of_lane(e, 63);
            exponent += end;
            const bool extreme = d != 0.f && !(fabsf(d) >= 0x1p-60f && fabsf(d) <= 0x1p60f);
            const bool wide = __any(!(fabs(e - mid) <= 60.0) || extreme);
            of.tail[lane] = power2(end - e) * d;
            if constexpr (FULL) {
                f.L[lane] = e;
                f.step[lane] = d;
                f.row[lane] = power2(e - mid);
                f.col[lane] = power2(mid - e) * d;
                of.up[lane] = power2(e);
            }
            if (lane == 0) {
                of.total = power2(end);
                of.wide = wide;
                of.bad = bads ? __builtin_ctzll(bads) : NEVER;
            }
        };

        if (tid < WAVES * CW)
            badcol[tid] = NEVER;
        if (tid < 2)
            badb[tid] = NEVER;

        // ---- The state before the segment. Column p of a tile (of lane c) is
        // row p of S; a lane has 4 rows n of each of 2 KN tiles, which
        // interleave, so that a pair of them is 8 adjacent n.
        f32x4 S[2 * KN];
        // each(S, pointer) for what there is of the state at s, by pieces of four. (The lane's number is made anew, or
        // the addresses of the first visit would be kept through the chunks for the last.)
        auto visit = [&](const float *s, int64_t index, auto each) __attribute__((always_inline)) {
            int l = lane;
            asm volatile("" : "+v"(l));
            const int gg = l >> 4, cc = l & 15;
            const float *base = s + (index * p.H + h) * p.P * p.N;
            const int row = col0 + cc;
            if (row < p.P) {
#pragma unroll
                for (int nt = 0; nt < 2 * KN; ++nt) {
                    const int n = 32 * (nt >> 1) + 8 * gg + 4 * (nt & 1);
                    if (n < p.N)
                        each(S[nt], base + (int64_t)row * p.N + n, p.N - n);
                }
            }
        };
        auto read4 = [&](const float *s, int left) __attribute__((always_inline)) {
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
            if constexpr (VEC) {
                v = *reinterpret_cast<const f32x4 *>(s);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < left)
                        v[e] = s[e];
            }
            return v;
        };
        auto write_state = [&](float *s, int64_t index) __attribute__((always_inline)) {
            if (!mine)
                return;
            visit(s, index, [&](const f32x4 &v, const float *at_, int left) __attribute__((always_inline)) {
                float *to = const_cast<float *>(at_);
                if constexpr (VEC) {
                    *reinterpret_cast<f32x4 *>(to) = v;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < left)
                            to[e] = v[e];
                }
            });
        };
        // The workspace's states lie as the lanes hold them: whole lines at a time, nothing to compare.
        auto kept = [&](int k, int nt) __attribute__((always_inline)) {
            const int64_t at0 = (((int64_t)k * p.H + h) * a.slices + job % a.slices) * (2 * KN) + nt;
            return reinterpret_cast<f32x4 *>(a.states) + at0 * 64 + lane;
        };
        auto keep = [&](int k) __attribute__((always_inline)) {
            if (mine)
#pragma unroll
                for (int nt = 0; nt < 2 * KN; ++nt)
                    *kept(k, nt) = S[nt];
        };
        const int slot = p.state_in || p.state_out ? seq_slot(p.seq, tile.n) : -1;
        const int last_number = number - index + (whole > 0 ? (whole - 1) / a.seg : 0);
        bool held = false;          // whether S may hold anything
#pragma unroll
        for (int nt = 0; nt < 2 * KN; ++nt)
            S[nt] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (index == 0 && (!FULL || last)) {
            if (p.state_in && slot >= 0) {
                held = true;
                visit(p.state_in, slot, [&](f32x4 &v, const float *s, int left) __attribute__((always_inline)) {
                    v = read4(s, left);
                });
            }
            // A sequence of several segments: its own state, which the call may
            // overwrite, is kept in the place of the one that the last segment
            // does not leave.
            if (!FULL)
                keep(last_number);
        } else if (FULL) {
            held = true;
            const int from = a.joined ? number : index == 0 ? last_number : number - index;
#pragma unroll
            for (int nt = 0; nt < 2 * KN; ++nt)
                S[nt] = *kept(from, nt);
#pragma unroll 2
            for (int k = a.joined ? number : number - index + 1; k < number; ++k) {
                const float by = a.decays[(int64_t)k * p.H + h];
#pragma unroll
                for (int nt = 0; nt < 2 * KN; ++nt) {
                    const f32x4 v = *kept(k, nt);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        S[nt][e] = fmaf(by, S[nt][e], v[e]);
                }
            }
        }

        if (chunks > 0) {
            load_step(0);
#pragma unroll
            for (int k = 0; k < LOADS; ++k)
                load(0, k);
            make_factors(0);
            load_step(1);
        }
        // The head whose M this wave has a share of (there are 1, 2 or 4 a workgroup, or fewer at a group's end), and its skip.
        const int mh = w & (a.heads - 1);
        float skip = 0.f;
        if (FULL && p.skip && mh < heads)
            skip = p.skip[group * per + head0 + mh];
        lds_barrier();              // the notes are set
        for (int ch = 0; ch < chunks; ++ch) {
            const int rows = min(len - ch * Q, Q);
            // The lane's place is made anew: addresses and comparisons that follow from it are cheaper made again than
            // kept from chunk to chunk (in spilled registers: 87 of them).
            asm volatile("" : "+v"(tid), "+s"(w));
            lane = tid & 63;
            g = lane >> 4;
            c = lane & 15;
            asm("" : "+v"(xo), "+v"(bo), "+v"(co), "+v"(go));
            put_bc(ch);
            put_x(ch);
            const bool wide = FULL && __builtin_amdgcn_readfirstlane(factors[mh].of[ch & 1].wide) != 0;
            lds_barrier();
            if (tid == 0)
                badb[(ch + 1) & 1] = NEVER;     // last read before the barrier that ended the chunk before
            f32x4 acc[4];
            if constexpr (FULL) {
                // M^T's blocks: tokens i of tile `it` as columns, 32 tokens j of step s as rows, two interleaving
                // tiles, so that a lane has 8 adjacent j of one i: an operand of the product with X.
                // Blocks (1,0) (2,0) (3,0) (0,0) (3,1) (2,1) go round the waves of a head.
                const Factors &fm = factors[mh];
                for (int f = mh < heads ? w / a.heads : MFRAGS; f < MFRAGS; f += WAVES / a.heads) {
                    const int it = f < 3 ? f + 1 : f == 3 ? 0 : 7 - f, s = f >= 4;
                    const int ti = 16 * it + c, tj0 = 32 * s + 8 * g;
                    const uint8_t *const c0 = cs + c_place(ti, g);
                    const uint8_t *const b0 = bs + b_place(32 * s + 8 * (c >> 2) + (c & 3), g);
                    const float r = fm.row[ti];
                    float col[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        col[e] = fm.col[tj0 + e];
                    f32x4 raw[2];
                    raw[0] = raw[1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int ks = 0; ks < KN; ++ks) {
                        bf16x8 cf[XP], bf[XP];
#pragma unroll
                        for (int i = 0; i < XP; ++i)
                            cf[i] = *reinterpret_cast<const bf16x8 *>(c0 + i * CBYTES + c_place(0, 4 * ks));
#pragma unroll
                        for (int tj = 0; tj < 2; ++tj) {
#pragma unroll
                            for (int i = 0; i < XP; ++i)
                                bf[i] = *reinterpret_cast<const bf16x8 *>(b0 + i * BBYTES + b_place(4 * tj, 4 * ks));
                            raw[tj] = product(bf, cf, raw[tj]);
                        }
                    }
                    // (The factors first: under a decay they come to d_j at most, where c . b times one of them may leave
                    // fp32's range or fall among its subnormal numbers.)
                    float m[8];
                    if (!wide) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            m[e] = raw[e >> 2][e & 3] * (col[e] * r);
                    } else {
                        const double Li = fm.L[ti];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            m[e] = raw[e >> 2][e & 3] * (fm.step[tj0 + e] * power2(Li - fm.L[tj0 + e]));
                    }
                    if (it >> 1 == s) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            m[e] = tj0 + e <= ti ? m[e] : 0.f;
                            m[e] = tj0 + e == ti ? m[e] + skip : m[e];
                        }
                    }
                    bf16x8 part[3];
                    split8(m, part);
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        reinterpret_cast<bf16x8 *>(xm + ((mh * MFRAGS + f) * 3 + i) * FRAG)[lane] = part[i];
                }

                // Y^T: S C^T.
#pragma unroll
                for (int it = 0; it < 4; ++it)
                    acc[it] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (held) {
                    const uint8_t *const c0 = cs + c_place(c, g);
#pragma unroll
                    for (int ks = 0; ks < KN; ++ks) {
                        bf16x8 sp[3];
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            v[e] = S[2 * ks + (e >> 2)][e & 3];
                        split8(v, sp);
#pragma unroll
                        for (int it = 0; it < 4; ++it) {
                            bf16x8 cf[XP];
#pragma unroll
                            for (int i = 0; i < XP; ++i)
                                cf[i] = *reinterpret_cast<const bf16x8 *>(c0 + i * CBYTES + c_place(16 * it, 4 * ks));
                            acc[it] = product(sp, cf, acc[it]);
                        }
                    }
                }
                lds_barrier();
            }
            const auto &f = factors[hi].of[ch & 1];
            const int bad_all = min(f.bad, badb[ch & 1]);
            const bool bad = bad_all != NEVER || __any(badcol[w * CW + (lane & (CW - 1))] != NEVER);
            if constexpr (FULL) {
                // Y^T: M X on top, then the gate, for all tiles at once: a branch inside would keep each tile's latencies
                // apart.
                const uint8_t *const ms = xm + hi * MFRAGS * 3 * FRAG + lane * 16;
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    const float up = f.up[16 * it + c];
                    acc[it] *= up;
#pragma unroll
                    for (int s = 0; s <= it >> 1; ++s) {
                        // Block (it, s) is number 0 1 2 4 for (1,0) (2,0) (3,0) (3,1), 3 for (0,0) and 5 for (2,1).
                        const int fr = it == 0 ? 3 : s == 0 ? it - 1 : it == 3 ? 4 : 5;
                        bf16x8 mf[3];
#pragma unroll
                        for (int i = 0; i < 3; ++i)
                            mf[i] = *reinterpret_cast<const bf16x8 *>(ms + (fr * 3 + i) * FRAG);
                        acc[it] = product(xf[s], mf, acc[it]);
                    }
                }
                if (p.gate) {
#pragma unroll
                    for (int it = 0; it < 4; ++it)
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            acc[it][e] *= silu(load_as_f32(&gate[it].v[e]));
                }
                if (bad) {
#pragma unroll
                    for (int it = 0; it < 4; ++it)
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            if (16 * it + c >= min(bad_all, badcol[w * CW + V * g + e]))
                                acc[it][e] = NAN;
                }
                T *yb = yp + (int64_t)ch * Q * p.yst;
                const auto yr = view(yb, p.yst, mine ? rows : 1, mine ? cols : 0);
                const uint32_t yo = offset_of(c, V * g, p.yst, cols);
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    // Columns V g + .. of token 16 it + c.
                    Gate o;
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        store_rne(&o.v[e], acc[it][e]);
                    const int t = 16 * it + c;
                    if constexpr (VEC) {
                        const uint32_t at0 = yo + it * (16 * (int)sizeof(T)) * (int)p.yst;
                        if constexpr (sizeof(Gate) == 16)
                            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o), yr, at0, 0, 0);
                        else
                            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, o), yr, at0, 0, 0);
                    } else if (mine && t < rows) {
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            if (V * g + e < cols)
                                yb[t * p.yst + V * g + e] = o.v[e];
                    }
                }
            }
            if (ch + 1 < chunks)
                make_factors(ch + 1);
            load_step(ch + 2);

            // S' = total S + B^T (tail x).
            const float total = f.total;
            const uint8_t *const b0 = bs + b_place(8 * g + (c >> 2), c & 3);
#pragma unroll
            for (int nt = 0; nt < 2 * KN; ++nt)
                S[nt] = held ? S[nt] * total : S[nt];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                bf16x8 xw[3];
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float x = (float)xf[s][0][e];
                    if constexpr (F32)
                        x = x + (float)xf[s][1][e] + (float)xf[s][2][e];
                    v[e] = x * f.tail[32 * s + 8 * g + e];
                }
                split8(v, xw);
#pragma unroll
                for (int nt = 0; nt < 2 * KN; ++nt) {
                    // The next chunk's loads, spread over these products.
                    const int step = s * 2 * KN + nt;
#pragma unroll
                    for (int k = step * LOADS / (4 * KN); k < (step + 1) * LOADS / (4 * KN); ++k)
                        load(ch + 1, k);
                    bf16x8 bt[XP];
#pragma unroll
                    for (int i = 0; i < XP; ++i) {
                        const uint8_t *const at0 = b0 + i * BBYTES + b_place(32 * s, 4 * (nt >> 1)) + 8 * (nt & 1);
                        bt[i] = join(transposed(at0), transposed(at0 + b_place(4, 0)));
                    }
                    S[nt] = product(bt, xw, S[nt]);
                }
            }
            held = true;
            if (bad) {
                if (bad_all != NEVER || badcol[w * CW + c] != NEVER)
#pragma unroll
                    for (int nt = 0; nt < 2 * KN; ++nt)
                        S[nt] = f32x4{NAN, NAN, NAN, NAN};
                if (lane < CW)
                    badcol[w * CW + lane] = NEVER;
            }
            lds_barrier();
        }
        if (FULL && last && p.state_out && slot >= 0)
            write_state(p.state_out, slot);
        if (!FULL) {
            keep(number);
            if (w < heads && lane == 0)
                a.decays[(int64_t)number * p.H + fh] = power2(exponent);
        }
    }
};

// bf16: eight waves of 16 columns; four a SIMD, from two workgroups, where the
// registers allow. fp32, whose operands take three times the LDS: four waves.
template <class T>
constexpr int WAVES = std::is_same<T, float>::value ? 4 : 8;

template <class T, int KN, bool FULL, bool VEC>
__global__ __launch_bounds__(64 * WAVES<T>)
    __attribute__((amdgpu_waves_per_eu(std::is_same<T, float>::value ? 1 : KN > 4 ? 2 : 4))) void heads_chunk_kernel(HeadsArgs a)
{
    Chunks<T, KN, WAVES<T>, FULL, VEC>::run(a);
}

// From the states that segments leave to those before them, along each sequence
// of several segments: a thread takes four states of one lane of the kernels
// above, eight segments at a time, their loads in flight together (32 segments of
// 32 heads of 64 x 64: 9.8 us, with four at a time and four waves a workgroup 11.7).
__global__ __launch_bounds__(NT_JOIN) void heads_join_kernel(HeadsArgs a, int per_head)
{
    const int64_t per = (int64_t)a.p.H * per_head;
    const int64_t i = (int64_t)blockIdx.x * NT_JOIN + threadIdx.x;
    if (i >= per)
        return;
    const int h = (int)(i / per_head);
    f32x4 *const states = reinterpret_cast<f32x4 *>(a.states) + i;
    for (int n = blockIdx.y; n < a.p.seq.num_seqs; n += gridDim.y) {
        const int64_t begin = seq_begin(a.p.seq, n), len = seq_begin(a.p.seq, n + 1) - begin;
        if (len <= a.seg)
            continue;
        const int64_t first = begin / a.seg + n, last = first + (len - 1) / a.seg;
        f32x4 v = states[first * per];
        states[first * per] = states[last * per];       // the sequence's own state
        for (int64_t k = first + 1; k <= last; k += 8) {
            f32x4 add[8];
            float by[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t at = k + j < last ? k + j : last;
                add[j] = states[at * per];
                by[j] = a.decays[at * a.p.H + h];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k + j <= last) {
                    states[(k + j) * per] = v;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = fmaf(by[j], v[e], add[j][e]);
                }
        }
    }
}

constexpr int LDS_MOST = 160 * 1024;

// How a call is laid out: everything that follows from its sizes alone.
struct Plan {
    int kn, slices, jobs, wgs, heads, seg;
    int64_t numbers;        // segments, numbered as in sequences.h
    bool parts;             // segments are shorter than a sequence may be
    bool joined;            // a sequence may have more than FOLDED of them
};

// Heads that `jobs` slices in a row may belong to, as a power of two.
int most_heads(int jobs, int slices)
{
    const int most = slices % jobs == 0 ? 1 : jobs % slices == 0 ? jobs / slices : (jobs - 2) / slices + 2;
    int n = 1;
    while (n < most)
        n *= 2;
    return n;
}

int lds_bytes(bool f32, int kn, int heads)
{
    if (f32)
        return kn == 2 ? Chunks<float, 2, WAVES<float>, true, true>::lds(heads)
                       : Chunks<float, 4, WAVES<float>, true, true>::lds(heads);
    return kn == 2   ? Chunks<uint16_t, 2, WAVES<uint16_t>, true, true>::lds(heads)
           : kn == 4 ? Chunks<uint16_t, 4, WAVES<uint16_t>, true, true>::lds(heads)
                     : Chunks<uint16_t, 8, WAVES<uint16_t>, true, true>::lds(heads);
}

bool make_plan(const Sequences &s, int H, int P, int groups, int N, conv_dtype dtype, Plan *l)
{
    const bool f32 = dtype == CONV_F32;
    // (64 rows of B and C of 256 states in three parts each would be 200 KB of LDS. Such prompts in fp32 go token by token:
    // 4096 tokens of 32 heads of 64 x 256 in 2410 us, in bf16 by chunks in 85.)
    if (N > (f32 ? 128 : 256))
        return false;
    l->kn = N <= 64 ? 2 : N <= 128 ? 4 : 8;
    l->slices = (P + 15) / 16;
    l->jobs = f32 ? WAVES<float> : WAVES<uint16_t>;
    l->heads = most_heads(l->jobs, l->slices);
    while (lds_bytes(f32, l->kn, l->heads) > LDS_MOST) {
        l->jobs /= 2;
        l->heads = most_heads(l->jobs, l->slices);
    }
    const int64_t group_jobs = (int64_t)(H / groups) * l->slices;
    if (group_jobs > (1 << 22))
        return false;
    l->wgs = (int)((group_jobs + l->jobs - 1) / l->jobs);
    // No segments where each compute unit has a workgroup without them: one prompt of 4096 tokens of 256 heads of 128 x
    // 128 (256 workgroups) takes 449 us whole and 456 in two, 4095 tokens of 512 heads of 64 x 128 in six prompts 415 and
    // 419. Otherwise segments such that some 512 workgroups have one (16384 tokens of 32 heads of 64 x 64: 122 us, with
    // 256 148, with 1024 135; 8192 tokens of 128 heads of 64 x 128: 264, 341 and 287), but at most 64 to the longest
    // sequence there can be (the first of these in 16: 148), and none of less than 256 tokens. (Whole calls.)
    const int64_t longest = s.offsets ? s.tokens : s.each;
    const int64_t whole = (int64_t)l->wgs * groups;      // workgroups without segments
    int64_t seg = whole * (s.offsets ? 1 : s.num_seqs) >= 256 ? longest : s.tokens * whole / 512;
    seg = seg > longest / 64 ? seg : longest / 64;
    seg = seg > 256 ? seg : 256;
    seg = (seg + Q - 1) / Q * Q;
    l->parts = seg < longest;
    l->joined = (longest + seg - 1) / seg > FOLDED;
    if (!l->parts)
        seg = (longest + Q) / Q * Q;
    if (seg > (1 << 30))
        return false;
    l->seg = (int)seg;
    l->numbers = seq_tiles(s, l->seg);
    // Threads of the grid below 2^32: 512 of them a workgroup in bf16, 256 in fp32.
    const int64_t threads = 64 * (f32 ? WAVES<float> : WAVES<uint16_t>);
    return (l->numbers * groups + 7) / 8 * 8 * l->wgs < (int64_t(1) << 32) / threads;
}

// Floats of the workspace's states, as the lanes hold them.
int64_t state_floats(const Plan &l, int H) { return l.numbers * H * l.slices * 16 * (32 * l.kn); }

int64_t space(const Plan &l, int H)
{
    return l.parts ? (state_floats(l, H) + (l.numbers * H + 63) / 64 * 64) * 4 : 0;
}

template <class T, int KN, bool FULL, bool VEC>
hipError_t launch_pass(const HeadsArgs &a, hipStream_t s)
{
    const hipError_t e = allow_lds<heads_chunk_kernel<T, KN, FULL, VEC>>(LDS_MOST);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL((heads_chunk_kernel<T, KN, FULL, VEC>), dim3((unsigned)((a.units + 7) / 8 * 8 * a.wgs)),
                       dim3(64 * WAVES<T>), (Chunks<T, KN, WAVES<T>, FULL, VEC>::lds(a.heads)), s, a);
    return hipGetLastError();
}

template <class T, int KN>
hipError_t launch(const HeadsArgs &a, bool parts, bool vec, hipStream_t s)
{
    if (parts) {
        const hipError_t e = vec ? launch_pass<T, KN, false, true>(a, s) : launch_pass<T, KN, false, false>(a, s);
        if (e != hipSuccess)
            return e;
    }
    if (a.joined) {
        const int per_head = a.slices * 2 * KN * 64;
        const int64_t blocks = ((int64_t)a.p.H * per_head + NT_JOIN - 1) / NT_JOIN;
        const int seqs = a.p.seq.num_seqs < 64 ? a.p.seq.num_seqs : 64;
        hipLaunchKernelGGL(heads_join_kernel, dim3((unsigned)blocks, (unsigned)seqs), dim3(NT_JOIN), 0, s, a, per_head);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return vec ? launch_pass<T, KN, true, true>(a, s) : launch_pass<T, KN, true, false>(a, s);
}

}  // namespace

bool heads_chunked_supports(int64_t tokens, int num_seqs, int H, int P, int groups, int N, conv_dtype dtype)
{
    Plan l;
    return make_plan(sequences_of(tokens, num_seqs, false), H, P, groups, N, dtype, &l) &&
           make_plan(sequences_of(tokens, num_seqs, true), H, P, groups, N, dtype, &l);
}

int64_t heads_chunked_workspace(int64_t tokens, int num_seqs, int H, int P, int groups, int N, conv_dtype dtype)
{
    Plan packed, equal;         // the larger of the two ways in which the sequences may lie
    make_plan(sequences_of(tokens, num_seqs, false), H, P, groups, N, dtype, &packed);
    make_plan(sequences_of(tokens, num_seqs, true), H, P, groups, N, dtype, &equal);
    const int64_t x = space(packed, H), y = space(equal, H);
    return x > y ? x : y;
}

hipError_t launch_heads_chunked(const HeadScanProblem &p, hipStream_t s)
{
    Plan l;
    make_plan(p.seq, p.H, p.P, p.groups, p.N, p.dtype, &l);
    HeadsArgs a;
    a.p = p;
    a.states = static_cast<float *>(p.workspace);
    a.decays = a.states + state_floats(l, p.H);
    a.seg = l.seg;
    a.units = (int)(l.numbers * p.groups);
    a.slices = l.slices;
    a.jobs = l.jobs;
    a.wgs = l.wgs;
    a.heads = l.heads;
    a.joined = l.joined;
    const int64_t e = p.dtype == CONV_F32 ? 4 : 2;
    const uintptr_t strides = (uintptr_t)((p.xst | p.xsh | p.yst | p.ysh | p.bst | p.bsg | p.cst | p.csg) * e) |
                              (p.gate ? (uintptr_t)((p.gst | p.gsh) * e) : 0);
    const uintptr_t at = (uintptr_t)p.x | (uintptr_t)p.y | (uintptr_t)p.b | (uintptr_t)p.c | (uintptr_t)p.gate |
                         (uintptr_t)p.state_in | (uintptr_t)p.state_out;
    const int64_t far = int64_t(1) << 22;       // 64 rows stay below 2^30 bytes
    auto rows_fit = [&](int64_t stride, int width) { return stride >= width && stride < far; };
    const bool vec = (strides | at) % 16 == 0 && p.P % (16 / e) == 0 && p.N % (16 / e) == 0 && rows_fit(p.xst, p.P) &&
                     rows_fit(p.yst, p.P) && rows_fit(p.bst, p.N) && rows_fit(p.cst, p.N) && (!p.gate || rows_fit(p.gst, p.P));
    if (p.dtype == CONV_F32)
        return l.kn == 2 ? launch<float, 2>(a, l.parts, vec, s) : launch<float, 4>(a, l.parts, vec, s);
    return l.kn == 2   ? launch<uint16_t, 2>(a, l.parts, vec, s)
           : l.kn == 4 ? launch<uint16_t, 4>(a, l.parts, vec, s)
                       : launch<uint16_t, 8>(a, l.parts, vec, s);
}

}  // namespace convfwd
