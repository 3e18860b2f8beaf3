// Norms of queries and keys for each head, and their rotation by position.
//
//   n_j = x_j rsqrt(mean_j x_j^2 + eps) w_j        (x_j itself without a weight)
//   (a, b) -> scale (a cos t - b sin t, b cos t + a sin t),  t = position * frequency
// for the pairs of a head's first R values; the others stay n_j.
//
// The bytes are the time: one pass, a head in the registers of L neighbouring
// lanes from its load to its store. A lane's unit is two pieces of V values
// that hold V whole pairs, i and i + R/2 or 2i and 2i + 1, so that no value
// changes lanes; the norm is an exchange between L lanes. V is the most that
// 16 bytes hold, where the sizes, strides and addresses allow.
//
// A workgroup takes `toks` tokens. Its threads first write their cosines and
// sines to LDS, one angle a thread (a token's 32 to 48 heads would make each of
// them as often, at some 60 instructions), then groups of L lanes go over the
// heads, `toks` groups side by side on one token each. 16384 tokens of 32 and 8
// heads of 128, bf16, with norms: 65 us, 0.34 GB at 5.15 TB/s (a plain copy:
// 5.1). 8 tokens: 5.2 to 5.9 us, of which a launch is 3: a thread's position, its
// frequency, the heads behind the barrier and the weights behind the norm's sum
// come one after the other.
//
// An angle is position times frequency, exact where that fits a double (29 bits
// of position times 24 of frequency, or more of the one and fewer of the other),
// else rounded to its 53 bits. It is reduced by quarters of a turn, pi / 2 in two
// parts of 53 bits each, up to 2^48 radians, and then held in fp32 to 2^-25 of a
// radian; the series of sine and cosine leave out less than 2^-28.
#include "common.h"
#include "eight_bit.h"
#include "internal.h"
#include "lanes.h"

namespace convfwd {
namespace {

constexpr int NT = 256;
constexpr int BATCH = 4;        // heads in flight a lane

__device__ __forceinline__ void turn(double position, float frequency, float scale, float &c, float &s)
{
    const double t = position * (double)frequency;
    const double q = rint(t * 0.63661977236758134308);
    const double r = fma(-q, 6.12323399573676603587e-17, fma(-q, 1.57079632679489661923, t));
    // (Past 2^48 the quarters are no longer exact: the angle is arbitrary, but no larger than the series are for.)
    const float x = fabs(r) > 1.0 ? 0.f : (float)r, z = x * x;
    float sn = 1.f / 362880.f;
    sn = fmaf(sn, z, -1.f / 5040.f);
    sn = fmaf(sn, z, 1.f / 120.f);
    sn = fmaf(sn, z, -1.f / 6.f);
    sn = fmaf(x * z, sn, x);
    float cs = -1.f / 3628800.f;
    cs = fmaf(cs, z, 1.f / 40320.f);
    cs = fmaf(cs, z, -1.f / 720.f);
    cs = fmaf(cs, z, 1.f / 24.f);
    cs = fmaf(cs, z, -0.5f);
    cs = fmaf(cs, z, 1.f);
    // The quarter, 0 to 3 (a NaN or infinite angle leaves NaN in x).
    const int k = (int)(q - 4.0 * floor(0.25 * q));
    c = scale * (k == 0 ? cs : k == 1 ? -sn : k == 2 ? -cs : sn);
    s = scale * (k == 0 ? sn : k == 1 ? cs : k == 2 ? -sn : -cs);
}

template <class T, int V>
struct Piece {
    T v[V] __attribute__((aligned(V * sizeof(T))));
};

template <class T, int V>
__device__ __forceinline__ Piece<T, V> load_piece(const T *p)
{
    Piece<T, V> t;
    __builtin_memcpy(&t, __builtin_assume_aligned(p, V * sizeof(T)), sizeof(t));
    return t;
}

// STREAM: past the caches, for outputs that would push each other out of them.
template <bool STREAM, class T, int V>
__device__ __forceinline__ void store_piece(T *p, const Piece<T, V> &t)
{
    if constexpr (V > 1 && STREAM) {
        typedef uint32_t Words __attribute__((ext_vector_type(V * sizeof(T) / 4)));
        __builtin_nontemporal_store(__builtin_bit_cast(Words, t), reinterpret_cast<Words *>(p));
    } else {
        __builtin_memcpy(__builtin_assume_aligned(p, V * sizeof(T)), &t, sizeof(t));
    }
}

struct RotaryArgs {
    RotaryProblem p;
    int toks;               // tokens of a workgroup
    int heads;              // heads of a workgroup
};

// L lanes a head, NU units of two pieces of V values a lane.
template <class T, int V, int L, int NU, bool INTER, bool STREAM>
__global__ __launch_bounds__(NT) void rotary_kernel(RotaryArgs a)
{
    const RotaryProblem &p = a.p;
    extern __shared__ float table[];        // cosines, then sines: [toks][R / 2] each
    const int half = p.rotated / 2;
    float *cosines = table, *sines = table + a.toks * half;
    const int64_t first = (int64_t)blockIdx.x * a.toks;
    for (int i = threadIdx.x; i < a.toks * half; i += NT) {
        const int tok = i / half;
        if (first + tok < p.tokens) {
            const double position = p.wide ? (double)static_cast<const int64_t *>(p.positions)[first + tok]
                                           : (double)static_cast<const int32_t *>(p.positions)[first + tok];
            turn(position, p.frequencies[i - tok * half], p.scale, cosines[i], sines[i]);
        }
    }
    __syncthreads();

    const int g = threadIdx.x / L, l = threadIdx.x % L;
    const int tok = g % a.toks;
    const int64_t t = first + tok;
    if (t >= p.tokens)
        return;
    // A unit's places in a head, which of its pieces are there and which of its
    // pairs (the first and the second half of them) are rotated. Neighbouring
    // lanes' pieces are neighbours, for the first and for the second pieces.
    int at0[NU], at1[NU];
    bool has0[NU], has1[NU], turn0[NU], turn1[NU];
    float cs[NU][V], sn[NU][V];
    constexpr bool PIECES = INTER && V > 1;     // each piece holds whole pairs
    const int pieces = p.D / V, across = PIECES ? (pieces + 1) / 2 : ((p.D - p.rotated) / V + 1) / 2;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        const int unit = l + L * u;
        int pair0, pair1;                       // of the first and of the second half of the unit's pairs
        if (PIECES) {
            at0[u] = unit * V;
            at1[u] = at0[u] + across * V;
            turn0[u] = unit < across && at0[u] < p.rotated;
            turn1[u] = unit < across && at1[u] < p.rotated;
            pair0 = at0[u] / 2;
            pair1 = at1[u] / 2;
            has0[u] = unit < across;
            has1[u] = unit < across && at1[u] < p.D;
        } else {
            pair0 = unit * V;
            pair1 = pair0 + V / 2;
            turn0[u] = turn1[u] = pair0 < half;
            const int rest = unit - half / V;   // of the pieces that are not rotated
            at0[u] = turn0[u] ? (INTER ? 2 * pair0 : pair0) : p.rotated + rest * V;
            at1[u] = turn0[u] ? (INTER ? 2 * pair0 + V : pair0 + half) : p.rotated + (rest + across) * V;
            has0[u] = turn0[u] || rest < across;
            has1[u] = turn0[u] || (rest < across && at1[u] < p.D);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool second = 2 * i >= V && V > 1;
            const bool on = second ? turn1[u] : turn0[u];
            const int at = tok * half + (second ? pair1 + i - V / 2 : pair0 + i);
            cs[u][i] = on ? cosines[at] : 1.f;
            sn[u][i] = on ? sines[at] : 0.f;
        }
    }
    const bool qnorm = p.qweight != nullptr, knorm = p.kweight != nullptr;
    const int total = p.Hq + p.Hk;
    const int step = NT / L / a.toks;
    const int begin = (int)blockIdx.y * a.heads, end = min(begin + a.heads, total);
    for (int h0 = begin + g / a.toks; h0 < end; h0 += step * BATCH) {
        Piece<T, V> e[BATCH][NU][2];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int h = h0 + b * step;
            if (h < end) {
                const T *x = h < p.Hq ? static_cast<const T *>(p.q) + t * p.qst + h * p.qsh
                                      : static_cast<const T *>(p.k) + t * p.kst + (h - p.Hq) * p.ksh;
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    e[b][u][0] = load_piece<T, V>(x + (has0[u] ? at0[u] : 0));
                    e[b][u][1] = load_piece<T, V>(x + (has1[u] ? at1[u] : 0));
                }
            }
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int h = h0 + b * step;
            if (h >= end)
                break;
            float f[NU][2][V];
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    f[u][0][i] = has0[u] ? load_as_f32(&e[b][u][0].v[i]) : 0.f;
                    f[u][1][i] = has1[u] ? load_as_f32(&e[b][u][1].v[i]) : 0.f;
                }
            const bool query = h < p.Hq;
            if (query ? qnorm : knorm) {
                auto squares = [&](float by) {
                    float s = 0.f;
#pragma unroll
                    for (int u = 0; u < NU; ++u)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float x = by * f[u][0][i], y = by * f[u][1][i];
                            s = fmaf(x, x, s);
                            s = fmaf(y, y, s);
                        }
                    return lanes_sum<L>(s);
                };
                const float ms = squares(1.f) / (float)p.D + p.eps;
                float r, by = 1.f;
                if (ms >= 0x1p-96f && ms <= 0x1p120f) {
                    r = 1.f / sqrtf(ms);
                } else {
                    // Squares that leave fp32's range are made again of values brought near it; zeros stay zeros.
                    by = ms < 1.f ? 0x1p100f : 0x1p-80f;
                    const float again = squares(by) / (float)p.D + p.eps * by * by;
                    r = again == 0.f ? 0.f : 1.f / sqrtf(ms < 0.f ? ms : again);     // (a negative eps: NaN)
                }
                const T *w = static_cast<const T *>(query ? p.qweight : p.kweight);
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    const Piece<T, V> w0 = load_piece<T, V>(w + (has0[u] ? at0[u] : 0));
                    const Piece<T, V> w1 = load_piece<T, V>(w + (has1[u] ? at1[u] : 0));
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        f[u][0][i] = f[u][0][i] * by * r * load_as_f32(&w0.v[i]);
                        f[u][1][i] = f[u][1][i] * by * r * load_as_f32(&w1.v[i]);
                    }
                }
            }
            T *y = query ? static_cast<T *>(p.q_out) + t * p.qot + h * p.qoh
                         : static_cast<T *>(p.k_out) + t * p.kot + (h - p.Hq) * p.koh;
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                Piece<T, V> o[2];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (2 * i >= V && V > 1 ? turn1[u] : turn0[u]) {
                        // Pair i: value i of each piece, or values 2i and 2i + 1 of the two as one run.
                        float &x0 = INTER ? f[u][2 * i / V][2 * i % V] : f[u][0][i];
                        float &x1 = INTER ? f[u][(2 * i + 1) / V][(2 * i + 1) % V] : f[u][1][i];
                        const float y0 = fmaf(x0, cs[u][i], -(x1 * sn[u][i])), y1 = fmaf(x1, cs[u][i], x0 * sn[u][i]);
                        x0 = y0;
                        x1 = y1;
                    }
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    store_rne(&o[0].v[i], f[u][0][i]);
                    store_rne(&o[1].v[i], f[u][1][i]);
                }
                if (has0[u])
                    store_piece<STREAM>(y + at0[u], o[0]);
                if (has1[u])
                    store_piece<STREAM>(y + at1[u], o[1]);
            }
        }
    }
}

template <class T, int V, int L, int NU>
void launch_units(const RotaryProblem &p, hipStream_t s)
{
    RotaryArgs a;
    a.p = p;
    const int total = p.Hq + p.Hk, groups = NT / L;
    // Few of both: only as many heads a workgroup as it has groups, so that the
    // heads spread over the compute units.
    const bool few = p.tokens * (int64_t)total <= 4096;
    // One token a workgroup up to four workgroups a compute unit (32 + 8 heads of 128, bf16: 512 tokens 6.0 us with one, 6.4
    // with two, 7.9 with four, 1024 7.6, 8.3 and 9.2), then two, or four where the groups have less than a batch of heads
    // with two. 16 + 16 heads of 128, fp32, 16 groups: 1111 tokens 9.7, 9.5 and 10.7, 16384 94, 95 and 99; 16 + 2 heads
    // of 256, bf16, 16 groups: 4096 tokens 19.6, 18.3 and 16.2.
    // With few heads more, so that every group has one (3 heads of 128, 109226
    // tokens: 67 us with 4 tokens, 37 with 8), as far as the table is 16 KB; not
    // where there are few tokens too (1300 of 3 heads of 64: 3.8 us, so 5.2).
    a.toks = p.tokens <= 1024 ? 1 : 2 * total < BATCH * groups ? 4 : 2;
    while (!few && a.toks * total < groups && a.toks * 2 * p.rotated <= 4096)
        a.toks *= 2;
    a.heads = few ? groups : total;
    const dim3 grid((unsigned)((p.tokens + a.toks - 1) / a.toks), (unsigned)((total + a.heads - 1) / a.heads));
    const size_t lds = (size_t)a.toks * p.rotated * sizeof(float);
    // Outputs past 64 MB leave the caches before a reader comes: streaming
    // stores, 16384 tokens of 40 heads of 128 in 65 us against 72. Smaller ones
    // stay: 4096 tokens of 18 heads of 256, written where the call before
    // wrote, in 16 us, streamed in 21. (Buffers that are all out of the caches
    // would gain by streaming at any size: 40 MB 16 against 23.)
    const bool stream = V > 1 && p.tokens * total * p.D * (int64_t)sizeof(T) > (int64_t(64) << 20);
    if (p.interleaved && stream)
        hipLaunchKernelGGL((rotary_kernel<T, V, L, NU, true, V != 1>), grid, dim3(NT), lds, s, a);
    else if (p.interleaved)
        hipLaunchKernelGGL((rotary_kernel<T, V, L, NU, true, false>), grid, dim3(NT), lds, s, a);
    else if (stream)
        hipLaunchKernelGGL((rotary_kernel<T, V, L, NU, false, V != 1>), grid, dim3(NT), lds, s, a);
    else
        hipLaunchKernelGGL((rotary_kernel<T, V, L, NU, false, false>), grid, dim3(NT), lds, s, a);
}

// Whether pieces of V values hold whole pairs and lie where a load of V values may.
bool fits(const RotaryProblem &p, int V, int64_t esize)
{
    const int64_t bytes = V * esize;
    uintptr_t bits = (uintptr_t)p.q | (uintptr_t)p.q_out | (uintptr_t)((p.qst | p.qsh | p.qot | p.qoh) * esize) |
                     (uintptr_t)p.qweight | (uintptr_t)p.kweight;
    if (p.Hk)
        bits |= (uintptr_t)p.k | (uintptr_t)p.k_out | (uintptr_t)((p.kst | p.ksh | p.kot | p.koh) * esize);
    return bits % bytes == 0 && p.D % V == 0 && p.rotated % (p.interleaved ? V : 2 * V) == 0;
}

template <class T, int V>
void launch_pieces(const RotaryProblem &p, hipStream_t s)
{
    // Pairs of pieces; the pieces that are not rotated make pairs of their own, an odd one a unit alone.
    const int rotated = p.interleaved && V > 1 ? 0 : p.rotated / (2 * V);
    const int units = rotated + (p.D - 2 * V * rotated + 2 * V - 1) / (2 * V);
    if constexpr (V == 1) {
        units <= 64 ? launch_units<T, V, 64, 1>(p, s) : launch_units<T, V, 64, 4>(p, s);
    } else {
        if (units <= 4)
            launch_units<T, V, 4, 1>(p, s);
        else if (units <= 8)
            launch_units<T, V, 8, 1>(p, s);
        else if (units <= 16)
            launch_units<T, V, 16, 1>(p, s);
        else if (units <= 32)
            launch_units<T, V, 32, 1>(p, s);
        else if (units <= 64)
            launch_units<T, V, 64, 1>(p, s);
        else
            launch_units<T, V, 64, 2>(p, s);
    }
}

template <class T>
void launch(const RotaryProblem &p, hipStream_t s)
{
    constexpr int V = 16 / sizeof(T);
    if (fits(p, V, sizeof(T)))
        launch_pieces<T, V>(p, s);
    else if (fits(p, V / 2, sizeof(T)))
        launch_pieces<T, V / 2>(p, s);
    else if (sizeof(T) == 2 && fits(p, 2, sizeof(T)))
        launch_pieces<T, 2>(p, s);
    else
        launch_pieces<T, 1>(p, s);
}

}  // namespace

// At most 256 units of two values a head; a grid's threads stay below 2^32 and its second axis within 2^16.
bool rotary_supports(int64_t tokens, int heads, int D)
{
    return D <= 512 && tokens < (int64_t(1) << 24) && heads <= (1 << 17);
}

hipError_t launch_rotary(const RotaryProblem &p, hipStream_t s)
{
    if (p.dtype == CONV_BF16)
        launch<uint16_t>(p, s);
    else
        launch<float>(p, s);
    return hipGetLastError();
}

}  // namespace convfwd
