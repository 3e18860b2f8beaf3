// The selective scan with a decay for each channel and state, by tiles of 128
// tokens.
//
//   d = step(dt + bias);  h[n] = exp(d a[c,n]) h[n] + d x b[n]
//   y = (sum_n c[n] h[n] + skip x) silu(gate)
//
// What a token, channel and state cost is an exponential, four or five other
// vector instructions, and little memory; what has to be found is parallel work.
// A workgroup takes 64 / LN neighbouring channels of a sequence; a lane holds
// four states of one channel, LN lanes a channel, and each of its eight waves
// takes 16 tokens of a tile:
//   1. all threads: step sizes and d x, of each token and channel once, and b
//      and c, in fp32 into LDS
//   2. each wave from a state of zeros over its tokens: the state it adds, and
//      the decay of all of them, into LDS; the 16 x 4 decays stay in registers
//   3. each wave puts together the state before its tokens from the tile's and
//      the waves' before it, and runs over its tokens again for y, with the
//      decays it has kept; the last wave leaves the state after the tile
//   4. all threads: skip, gate and store.
// The second run costs three instructions a state where a second kernel (or a
// scan of a whole tile's pieces) would cost an exponential more.
//
// Where there are too few channels and sequences to fill the chip, sequences
// are cut into segments of `seg` tokens: a first kernel (steps 1 and 2 only)
// leaves the state each segment but the last adds, and its decay; the second
// one begins with the state put together from those before its segment. The
// first segment's initial state is kept in the place of the last one's, which
// leaves none, since the call may overwrite it in place.
//
// 8192 tokens of 8192 channels of 16 states, bf16: 439 us, 1.23 TB/s; vector
// instructions bound it. A token of a wave is 256 states, and takes a SIMD 257
// clocks. By the counters it is 46 vector instructions, issued in 206 of them:
// for each of a lane's four states an exponential, a product by the rate, twice
// a product with b, and three of the recurrence and y, 28 together; the other 18
// are step sizes, gates, conversions, sums over lanes and addresses. LDS is busy
// in half of the clocks, 6 % of them bank conflicts; the rest is the three
// barriers of a tile. Four waves and tiles of 64 tokens, with the products d x b
// kept, took 513 us.
//
// With 8 states and fewer a thread has eight channels in steps 1 and 4 beside the
// 64 decays, which then do not all stay in registers (10 go to memory in bf16, 24
// in fp32): 409 us for 8192 channels of 8 states in bf16, 705 in fp32, against
// 412 in fp32 for 16 states.
#include "common.h"
#include "eight_bit.h"
#include "internal.h"
#include "lanes.h"
#include "scan_math.h"
#include "sequences.h"

namespace convfwd {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int WAVES = 8;
constexpr int NT = 64 * WAVES;
constexpr int TS = 16;                  // tokens of a wave
constexpr int TILE = TS * WAVES;

struct ScanArgs {
    ScanProblem p;
    f32x4 *states, *decays;     // workspace: [segment number][slice][lane]
    int seg;                    // tokens of a segment, a multiple of TILE
    int numbers;                // segment numbers
    int slices;                 // slices of 64 / LN channels, none across two groups
    int group_slices;           // of a group
};

// A barrier for LDS traffic only: __syncthreads would also wait for the loads
// of the next tile that are in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// A thread's piece of a row: in fp32 eight values, 32 bytes, are two parts of 16.
template <class T, int V>
struct Piece {
    static constexpr int PART = V * sizeof(T) < 16 ? V : 16 / sizeof(T);
    T v[V] __attribute__((aligned(PART * sizeof(T))));
};

// How pieces are loaded and stored (a host rule): a value at a time, aligned
// parts, of which a row's last piece may have only some, or whole.
enum Pieces { VALUES, PARTS, WHOLE };

template <class T, int LN, bool FULL, Pieces VEC>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(4))) void scan_tile_kernel(ScanArgs a)
{
    constexpr int CH = 64 / LN, NP = 4 * LN;    // channels of a workgroup, states of a channel (padded)
    constexpr int EC = CH / 4;                  // channels of a thread's piece in steps 1 and 4: four threads a token
    constexpr int EB = TILE * NP / NT;          // states of a thread's piece of b, and of c: NP states a token
    const ScanProblem &p = a.p;
    __shared__ __align__(16) f32x2 steps[TILE][CH];     // d and d x; then y in d's place
    __shared__ __align__(16) float bs[TILE][NP], cs[FULL ? TILE : 1][NP];
    __shared__ f32x4 fold[WAVES][2][64];                // decay of a wave's tokens, state they add
    __shared__ f32x4 carry[64];                         // the state before the tile
    __shared__ __align__(16) float biases[CH], skips[CH];

    // Workgroup i runs on XCD i % 8: neighbouring channels, which share lines of x, go to one XCD.
    const int xcd = (int)blockIdx.x & 7, around = (a.slices + 7) / 8;
    const int slice = xcd * around + (int)(blockIdx.x >> 3) % around, number = (int)(blockIdx.x >> 3) / around;
    if (slice >= a.slices || number >= a.numbers)
        return;
    const SeqTile tile = seq_tile(p.seq, a.seg, number);
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
    const int tiles = (len + TILE - 1) / TILE;

    int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group_channels = p.channels / p.groups, group = slice / a.group_slices;
    const int begin = group * group_channels + slice % a.group_slices * CH, end = (group + 1) * group_channels;
    // In steps 2 and 3: channel and states of the lane.
    const int c = begin + lane / LN, n0 = 4 * (lane % LN);
    const bool live = c < end;
    // In steps 1 and 4: token and channels of the thread; its token and states of b and c.
    int tok = tid >> 2, ch0 = (tid & 3) * EC, cc = begin + ch0;
    int btok = tid * EB / NP, bn = tid * EB % NP;
    const T *xp = static_cast<const T *>(p.x) + first * p.xs, *dp = static_cast<const T *>(p.dt) + first * p.dts;
    const T *gp = p.gate ? static_cast<const T *>(p.gate) + first * p.gs : xp;
    const int64_t gs = p.gate ? p.gs : p.xs;
    const T *bp = static_cast<const T *>(p.b) + first * p.bst + group * p.bsg;
    const T *cp = static_cast<const T *>(p.c) + first * p.cst + group * p.csg;
    T *yp = static_cast<T *>(p.y) + first * p.ys;

    // Values past the channels (states) are the row's first ones, and are not used.
    auto row_piece = [&](auto &to, const T *row, int at, int width) __attribute__((always_inline)) {
        constexpr int V = sizeof(to.v) / sizeof(T), STEP = VEC == WHOLE ? V : Piece<T, V>::PART;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < V; i += STEP)
                __builtin_memcpy(to.v + i, __builtin_assume_aligned(row + (at + i < width ? at + i : 0), alignof(Piece<T, V>)),
                                 STEP * sizeof(T));
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                to.v[i] = row[at + i < width ? at + i : 0];
        }
    };
    Piece<T, EC> xv, dv, gv;
    Piece<T, EB> bv, cv;
    // A tile's rows lie within 2^31 bytes of its first one (VEC: a host rule): one address for all lanes, and a lane's
    // offset by one multiplication of 24 bits.
    auto row_of = [&](const T *base, int64_t stride, int t, int r) __attribute__((always_inline)) {
        base += (int64_t)t * TILE * stride;
        if constexpr (VEC)
            return reinterpret_cast<const T *>(reinterpret_cast<const char *>(base) +
                                               __umul24((uint32_t)r, (uint32_t)stride * (uint32_t)sizeof(T)));
        else
            return base + r * stride;
    };
    auto load = [&](int t) __attribute__((always_inline)) {
        const int rows = min(len - t * TILE, TILE);
        const int r = min(tok, rows - 1), rb = min(btok, rows - 1);
        row_piece(xv, row_of(xp, p.xs, t, r), cc, end);
        row_piece(dv, row_of(dp, p.dts, t, r), cc, end);
        row_piece(bv, row_of(bp, p.bst, t, rb), bn, p.N);
        if constexpr (FULL) {
            row_piece(gv, row_of(gp, gs, t, r), cc, end);
            row_piece(cv, row_of(cp, p.cst, t, rb), bn, p.N);
        }
    };
    if (tiles > 0)
        load(0);
    if (tid < CH) {
        const int ci = begin + tid < end ? begin + tid : begin;
        biases[tid] = p.bias ? p.bias[ci] : 0.f;
        skips[tid] = p.skip ? p.skip[ci] : 0.f;
    }

    // ---- The lane's rates and the state before the segment.
    const int64_t sat = (int64_t)(live ? c : 0) * p.N + n0;
    auto four = [&](const float *s) __attribute__((always_inline)) {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if constexpr (VEC) {
            if (live && n0 < p.N)
                v = *reinterpret_cast<const f32x4 *>(s);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (live && n0 + i < p.N)
                    v[i] = s[i];
        }
        return v;
    };
    // (Never minus infinity: times the zero step of a token that is not there it has to be zero.)
    f32x4 rate = four(p.a + sat);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        rate[i] = rate_of_log2(rate[i]);
    const int64_t state_size = (int64_t)p.channels * p.N;
    const int slot = p.state_in || p.state_out ? seq_slot(p.seq, tile.n) : -1;
    auto kept = [&](f32x4 *base, int k) { return base + ((int64_t)k * a.slices + slice) * 64 + lane; };
    const int first_number = number - index;
    const int last_number = first_number + (whole > 0 ? (whole - 1) / a.seg : 0);
    if (w == 0) {
        f32x4 h = {0.f, 0.f, 0.f, 0.f};
        if (index == 0 && (!FULL || last)) {
            if (p.state_in && slot >= 0)
                h = four(p.state_in + slot * state_size + sat);
            if (!FULL)
                *kept(a.states, last_number) = h;
        } else if (FULL) {
            h = *kept(a.states, index == 0 ? last_number : first_number);
#pragma unroll 4
            for (int k = first_number + 1; k < number; ++k)
                h = *kept(a.decays, k) * h + *kept(a.states, k);
        }
        carry[lane] = h;
    }

    lds_barrier();                  // biases and skips are there
    float total = 0.f;              // sum of the steps of the wave's tokens so far
    for (int t = 0; t < tiles; ++t) {
        const int rows = min(len - t * TILE, TILE);
        // The thread's place is made anew: addresses that follow from it are cheaper made again than kept from tile to
        // tile beside the decays (in spilled registers).
        asm volatile("" : "+v"(tid));
        lane = tid & 63;
        tok = tid >> 2;
        ch0 = (tid & 3) * EC;
        cc = begin + ch0;
        btok = tid * EB / NP;
        bn = tid * EB % NP;
        // ---- 1.
        const bool there = tok < rows;
        float x[EC], d[EC], dx[EC], bf[EB], cf[EB];
#pragma unroll
        for (int i = 0; i < EC; ++i) {
            x[i] = load_as_f32(&xv.v[i]);
            d[i] = step_size(load_as_f32(&dv.v[i]) + biases[ch0 + i], p.softplus);
            dx[i] = d[i] * x[i];
        }
#pragma unroll
        for (int i = 0; i < EB; ++i) {
            bf[i] = load_as_f32(&bv.v[i]);
            cf[i] = FULL ? load_as_f32(&cv.v[i]) : 0.f;
        }
        if (rows < TILE || p.N < NP) {      // zeros for what is not there
#pragma unroll
            for (int i = 0; i < EC; ++i)
                d[i] = there ? d[i] : 0.f, dx[i] = there ? dx[i] : 0.f;
#pragma unroll
            for (int i = 0; i < EB; ++i) {
                const bool in = btok < rows && bn + i < p.N;
                bf[i] = in ? bf[i] : 0.f;
                cf[i] = in ? cf[i] : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < EC; i += 2)
            *reinterpret_cast<f32x4 *>(&steps[tok][ch0 + i]) = f32x4{d[i], dx[i], d[i + 1], dx[i + 1]};
        auto put = [&](float *to, const float(&v)[EB]) __attribute__((always_inline)) {
            if constexpr (EB >= 4) {
#pragma unroll
                for (int i = 0; i < EB; i += 4)
                    *reinterpret_cast<f32x4 *>(to + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
            } else {
                *reinterpret_cast<f32x2 *>(to) = f32x2{v[0], v[1]};
            }
        };
        put(&bs[btok][bn], bf);
        if constexpr (FULL)
            put(&cs[btok][bn], cf);
        Piece<T, EC> gate = gv;
        lds_barrier();
        if (t + 1 < tiles)
            load(t + 1);
        // ---- 2.
        const int waves = (rows + TS - 1) / TS;         // that have tokens; the others have nothing to do here
        const f32x4 before = carry[lane];
        f32x4 e[TS];
        f32x4 h = {0.f, 0.f, 0.f, 0.f};
        float sum = 0.f;
        const f32x2 *st = &steps[TS * w][lane / LN];
        const f32x4 *bw = reinterpret_cast<const f32x4 *>(&bs[TS * w][n0]);
        if (w < waves) {
#pragma unroll
            for (int s = 0; s < TS; ++s) {
                const f32x2 v = st[s * CH];
                const f32x4 b = bw[s * LN];
                sum += v[0];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    e[s][i] = __builtin_amdgcn_exp2f(v[0] * rate[i]);
                    h[i] = fmaf(e[s][i], h[i], v[1] * b[i]);
                }
            }
            f32x4 all;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                all[i] = __builtin_amdgcn_exp2f(sum * rate[i]);
            fold[w][0][lane] = all;
            fold[w][1][lane] = h;
        }
        lds_barrier();
        // ---- 3.
        if (w < waves) {
            h = before;
            const int upto = FULL ? w : waves;
            if (FULL || w == waves - 1)
#pragma unroll
                for (int j0 = 0; j0 < (FULL ? WAVES - 1 : WAVES); j0 += 2)
                    if (j0 < upto) {            // two at a time, their reads in flight together
                        f32x4 pj[2], hj[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            pj[j] = fold[j0 + j][0][lane];
                            hj[j] = fold[j0 + j][1][lane];
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (j0 + j < upto)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    h[i] = fmaf(pj[j][i], h[i], hj[j][i]);
                    }
            if constexpr (FULL) {
                const f32x4 *cw = reinterpret_cast<const f32x4 *>(&cs[TS * w][n0]);
                // y of U tokens at a time: lane u of a channel ends with the sum for token u.
                constexpr int U = LN < 4 ? LN : 4;
                float *yw = reinterpret_cast<float *>(&steps[TS * w][lane / LN]) + (LN <= 4 || lane % LN < 4 ? lane % U * CH * 2 : 0);
#pragma unroll
                for (int s0 = 0; s0 < TS; s0 += U) {
                    float y[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int s = s0 + u;
                        const float dxs = st[s * CH][1];
                        const f32x4 b = bw[s * LN], ct = cw[s * LN];
                        y[u] = 0.f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            h[i] = fmaf(e[s][i], h[i], dxs * b[i]);
                            y[u] = fmaf(h[i], ct[i], y[u]);
                        }
                    }
                    float sum_u = lanes_scatter<U>(y, lane);
                    if constexpr (LN == 8)
                        sum_u += lane_moved<0x104>(sum_u);      // of the lane four above
                    if (LN <= 4 || lane % LN < 4)
                        yw[s0 * CH * 2] = sum_u;
                }
            }
        }
        total += sum;
        if (w == waves - 1)
            carry[lane] = h;
        lds_barrier();
        // ---- 4.
        if constexpr (FULL) {
            Piece<T, EC> o;
#pragma unroll
            for (int i = 0; i < EC; ++i) {
                float y = fmaf(skips[ch0 + i], x[i], steps[tok][ch0 + i][0]);
                if (p.gate)
                    y *= silu(load_as_f32(&gate.v[i]));
                store_rne(&o.v[i], y);
            }
            T *yr = const_cast<T *>(row_of(yp, p.ys, t, tok)) + cc;
            if (there) {
                if constexpr (VEC) {
                    constexpr int STEP = VEC == WHOLE ? EC : Piece<T, EC>::PART;
#pragma unroll
                    for (int i = 0; i < EC; i += STEP)
                        if (cc + i < end)
                            __builtin_memcpy(__builtin_assume_aligned(yr + i, alignof(Piece<T, EC>)), o.v + i, STEP * sizeof(T));
                } else {
#pragma unroll
                    for (int i = 0; i < EC; ++i)
                        if (cc + i < end)
                            yr[i] = o.v[i];
                }
            }
        }
    }
    if constexpr (!FULL)
        fold[w][0][lane][0] = total;
    lds_barrier();
    if (w != 0)
        return;
    const f32x4 h = carry[lane];
    if constexpr (FULL) {
        if (last && p.state_out && slot >= 0 && live) {
            float *to = p.state_out + slot * state_size + sat;
            if constexpr (VEC) {
                if (n0 < p.N)
                    *reinterpret_cast<f32x4 *>(to) = h;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n0 + i < p.N)
                        to[i] = h[i];
            }
        }
    } else {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < WAVES; ++j)
            sum += fold[j][0][lane][0];
        f32x4 all;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            all[i] = __builtin_amdgcn_exp2f(sum * rate[i]);
        *kept(a.states, number) = h;
        *kept(a.decays, number) = all;
    }
}

// How a call is laid out: everything that follows from its sizes alone.
struct Plan {
    int ln, group_slices, slices, seg;
    int64_t numbers;        // segments, numbered as in sequences.h
    bool parts;             // segments are shorter than a sequence may be
};

bool make_plan(const Sequences &s, int channels, int groups, int N, Plan *l)
{
    if (N > 32)         // more go token by token: 4096 tokens of 2048 channels of 64 states in 1700 us
        return false;
    l->ln = N <= 8 ? 2 : N <= 16 ? 4 : 8;
    l->group_slices = (channels / groups + 64 / l->ln - 1) / (64 / l->ln);
    if ((int64_t)l->group_slices * groups > (1 << 22))
        return false;
    l->slices = l->group_slices * groups;
    // No segments where each compute unit has a workgroup without them: one prompt of 8192 tokens and 6144 channels of 16
    // takes 439 us whole and 491 in segments, 2047 tokens of 4096 channels in six prompts 75 and 100; the least such
    // prompt, 4096 channels (256 workgroups), is the exception, 331 and 310. Otherwise segments such that some 1024
    // workgroups have one (2048 channels: 171 us, with 512 176, whole 304; 1024 channels 92, 92 and 298), but at most 16
    // to the longest sequence there can be, and none of less than 256 tokens.
    const int64_t longest = s.offsets ? s.tokens : s.each;
    int64_t seg = (int64_t)l->slices * (s.offsets ? 1 : s.num_seqs) >= 256 ? longest : s.tokens * l->slices / 1024;
    seg = seg > longest / 16 ? seg : longest / 16;
    seg = seg > 256 ? seg : 256;
    seg = (seg + TILE - 1) / TILE * TILE;
    l->parts = seg < longest;
    if (!l->parts)
        seg = (longest + TILE) / TILE * TILE;
    if (seg > (1 << 30))
        return false;
    l->seg = (int)seg;
    l->numbers = seq_tiles(s, l->seg);
    // Threads of the grid below 2^32.
    return l->numbers * ((l->slices + 7) / 8 * 8) < (int64_t(1) << 23);
}

// Bytes of the workspace's states, and of its decays.
int64_t half_space(const Plan &l) { return l.parts ? l.numbers * l.slices * 64 * 16 : 0; }

template <class T, int LN, Pieces VEC>
hipError_t launch_kernels(const ScanArgs &a, bool segments, hipStream_t s)
{
    const dim3 grid((unsigned)(a.numbers * ((a.slices + 7) / 8 * 8))), block(NT);
    if (segments) {
        hipLaunchKernelGGL((scan_tile_kernel<T, LN, false, VEC>), grid, block, 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL((scan_tile_kernel<T, LN, true, VEC>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <class T, int LN>
hipError_t launch_lanes(const ScanArgs &a, bool segments, bool vec, hipStream_t s)
{
    // A thread's piece: EC channels, or EB states of b and of c. Pieces that are one part are whole where parts are. A
    // prompt of 4096 tokens of 8 states, fp32: 8192 channels 346 us by whole pieces and some 7 % more by parts, 8188 374 by
    // parts, 8191 613 by values.
    constexpr int EC = 16 / LN, EB = LN;
    constexpr bool SPLIT = EC > Piece<T, EC>::PART || EB > Piece<T, EB>::PART;
    if (!vec)
        return launch_kernels<T, LN, VALUES>(a, segments, s);
    if (SPLIT && (a.p.channels / a.p.groups % EC != 0 || a.p.N % EB != 0))
        return launch_kernels<T, LN, SPLIT ? PARTS : WHOLE>(a, segments, s);
    return launch_kernels<T, LN, WHOLE>(a, segments, s);
}

template <class T>
hipError_t launch(const ScanArgs &a, const Plan &l, hipStream_t s)
{
    // A thread's piece: 16 / LN channels, or LN states of b and of c; of their parts, 16 bytes at most, a row has whole ones.
    const ScanProblem &p = a.p;
    const int64_t ec = 16 / l.ln * sizeof(T), eb = l.ln * sizeof(T);
    const uintptr_t rows = (uintptr_t)p.x | (uintptr_t)p.dt | (uintptr_t)p.gate | (uintptr_t)p.y |
                           (uintptr_t)((p.xs | p.dts | p.ys | (p.gate ? p.gs : 0)) * sizeof(T)) |
                           (uintptr_t)(p.channels / p.groups * sizeof(T));
    const uintptr_t bc = (uintptr_t)p.b | (uintptr_t)p.c | (uintptr_t)((p.bst | p.bsg | p.cst | p.csg) * sizeof(T)) |
                         (uintptr_t)(p.N * sizeof(T));
    const uintptr_t st = (uintptr_t)p.a | (uintptr_t)p.state_in | (uintptr_t)p.state_out;
    const int64_t far = int64_t(1) << 22;       // a row's bytes fit 24 bits
    const bool vec = p.xs < far && p.dts < far && p.ys < far && (!p.gate || p.gs < far) && p.bst < far && p.cst < far &&
                     rows % (ec < 16 ? ec : 16) == 0 && bc % (eb < 16 ? eb : 16) == 0 && st % 16 == 0 && p.N % 4 == 0;
    switch (l.ln) {
    case 2: return launch_lanes<T, 2>(a, l.parts, vec, s);
    case 4: return launch_lanes<T, 4>(a, l.parts, vec, s);
    default: return launch_lanes<T, 8>(a, l.parts, vec, s);
    }
}

}  // namespace

bool scan_tiled_supports(int64_t tokens, int num_seqs, int channels, int groups, int N)
{
    Plan l;
    return make_plan(sequences_of(tokens, num_seqs, false), channels, groups, N, &l) &&
           make_plan(sequences_of(tokens, num_seqs, true), channels, groups, N, &l);
}

int64_t scan_tiled_workspace(int64_t tokens, int num_seqs, int channels, int groups, int N)
{
    Plan packed, equal;         // the larger of the two ways in which the sequences may lie
    make_plan(sequences_of(tokens, num_seqs, false), channels, groups, N, &packed);
    make_plan(sequences_of(tokens, num_seqs, true), channels, groups, N, &equal);
    const int64_t x = half_space(packed), y = half_space(equal);
    return 2 * (x > y ? x : y);
}

hipError_t launch_scan_tiled(const ScanProblem &p, hipStream_t s)
{
    Plan l;
    make_plan(p.seq, p.channels, p.groups, p.N, &l);
    ScanArgs a;
    a.p = p;
    a.states = static_cast<f32x4 *>(p.workspace);
    a.decays = a.states + half_space(l) / 16;
    a.seg = l.seg;
    a.numbers = (int)l.numbers;
    a.slices = l.slices;
    a.group_slices = l.group_slices;
    return p.dtype == CONV_BF16 ? launch<uint16_t>(a, l, s) : launch<float>(a, l, s);
}

}  // namespace convfwd
