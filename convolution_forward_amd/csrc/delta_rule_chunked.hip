// The gated delta rule by chunks of 64 tokens on the matrix cores, bf16 or fp32
// operands, in fp32 precision.
//
// Inside a chunk let G_i be the sum of the gates up to token i, r_i the factor
// that normalises k_i (1 without), and S the state before the chunk. With
//   A_ij = beta_i r_i r_j exp(G_i - G_j) (k_i . k_j)   for j < i, else 0
//   P_ij = scale rq_i r_j exp(G_i - G_j) (q_i . k_j)   for j <= i, else 0
// the rule's 64 steps are
//   U  = (1 + A)^-1 diag(beta) (V - diag(r exp G) K S)
//   O  = diag(scale rq exp G) Q S + P U
//   S' = exp(G_63) S + K^T diag(r_i exp(G_63 - G_i)) U.
// No exponent is ever positive for gates <= 0, and differences of G are taken
// in 64 bits, so a strong gate early in a chunk costs the later ones nothing.
// exp is the instruction's after a product with log2 e: its error, |x| 2^-24 of
// the value, is that of rounding x itself to fp32.
//
// Two kernels. The first takes every chunk and key head at once and writes
// what does not depend on S: T = (1 + A)^-1 diag(beta), P, the row factors, and
// K and Q, all in the order in which the second one's matrix instructions take
// them. (K and Q read where they are, 64-byte pieces of 16 rows an instruction,
// cost the second kernel more than the copy costs the first: six prompts of
// 4096 tokens, 98 -> 117 us and 36 -> 34.) The second carries S along each
// sequence. Columns of S are independent, so a workgroup takes 16 of them; four
// of its waves share the rows. (32 columns halve the loads a column, and the
// workgroups: no faster, 103 us for the six prompts.)
//
// 16384 tokens of one prompt, 16 key and 32 value heads of 128 x 128: the first
// 112-117 us, 0.52 GB at 4.5 TB/s; the second 458-484 us, 256 chunks of 1.8-1.9
// us each, one workgroup a compute unit. There the chain of exchanges is most
// of the time, and the output waves, which share its SIMDs, the rest: their
// products of third parts cost 0.14 us a chunk. With two workgroups a compute
// unit a chunk of both takes 3 us.
//
// Precision, bf16: operands (K, Q) are exact, every other operand of a product
// is split into bf16 parts x = hi + mid + lo (each the nearest bf16 of what is
// left, 24 bits together), and the products of parts above 2^-24 are added in
// fp32: three for an exact operand times a split one, six for two split ones.
// fp32 operands go through the fp32 matrix instructions as they are.
//
// Values that are not finite: a zero of T or P times a NaN would carry it to
// earlier tokens. So rows of K that hold one are read as zeros, and so are
// values of V - .., of U and of a product on the way to T that are not finite
// or have overflowed, and the token is noted; from it on the outputs and the
// final state are set to NaN, for all columns (K, g, beta, T) or for its own
// (V, S, U).
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "sequences.h"

namespace convfwd {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr int C = 64;                   // tokens of a chunk
constexpr int NT = 256;
constexpr float UNIT_EPS = 1e-6f;
constexpr int NEVER = 0x7fffffff;

// Token (within the chunk) of row r of token tile i. Tiles 2s and 2s + 1
// interleave, so that a lane's four rows of each, as results leave the matrix
// cores, are eight adjacent tokens: the K order of the next product.
__device__ __forceinline__ int token_of(int i, int r) { return 32 * (i >> 1) + 8 * (r >> 2) + 4 * (i & 1) + (r & 3); }

// ---- Workspace ---------------------------------------------------------------
// For each chunk number and key head: K (wave, tile) and Q (tile, wave), 4 x 4
// fragments each. For each chunk number and value head: T, 3 parts of the 6
// fragments that are not all zero, P, the same 6 in fp32, two each, then 4 x 64
// row factors and a header. A fragment is 64 lanes x 16 bytes.
constexpr int FRAG = 1024;

// In fp32: K (wave, tile, d), Q (tile, wave, d) and K^T (wave, d, tile), 16 DT
// fragments each; T and P, 10 fragments each.
template <int DT, bool F32>
struct Space {
    static constexpr int Q = (F32 ? 16 * DT : 16) * FRAG, KT = 2 * Q, KEY = F32 ? 3 * Q : 2 * Q;
    static constexpr int P = (F32 ? 10 : 18) * FRAG, UPK = (F32 ? 20 : 30) * FRAG, UPQ = UPK + 256, TAIL = UPQ + 256,
                         HEAD = TAIL + 256;     // exp(G_63), first token that is not finite
    static constexpr int VAL = UPK + FRAG;
};

// Place of fragment (tile i, K step s) among the six of a lower triangle.
__device__ __forceinline__ int low_frag(int i, int s) { return i < 2 ? i : 2 * i - 2 + s; }

struct ChunkArgs {
    DeltaProblem p;
    uint8_t *keys, *vals;       // workspace
    int vec;                    // rows of q and k take 16-byte loads
    int heads;                  // value heads of a key head that a workgroup of the first kernel takes
    int slices;                 // column slices of a head
};

// A barrier for LDS traffic only: __syncthreads would also wait for the loads
// of the next chunk that are in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ __forceinline__ __bf16 part_of(float &x)
{
    const __bf16 h = (__bf16)x;
    x -= (float)h;
    return h;
}

template <int DT, bool F32>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(F32 ? 2 : 4))) void delta_prepare_kernel(ChunkArgs a)
{
    using W = Space<DT, F32>;
    using T = typename std::conditional<F32, float, uint16_t>::type;
    constexpr int D = 64 * DT, E = 16 / sizeof(T), PITCH = D + E, MP = 68;
    const DeltaProblem &p = a.p;
    // K and Q give their room to A (then T) and P once their products are in registers.
    constexpr int KROWS = C * PITCH * (int)sizeof(T), ROWS = KROWS > C * MP * 4 ? KROWS : C * MP * 4;
    __shared__ __align__(16) uint8_t room[2 * ROWS];
    T *ks = reinterpret_cast<T *>(room), *qs = reinterpret_cast<T *>(room + ROWS);
    float *m = reinterpret_cast<float *>(room), *pm = reinterpret_cast<float *>(room + ROWS);
    // Four 16x16 blocks between the two halves of the last inversion step, in a corner of m that nothing else uses.
    auto z = [&](int i) { return m + 16 * (i >> 1) * MP + 32 + 16 * (i & 1); };
    __shared__ __align__(16) double gs[4][C];      // of up to four value heads at a time
    __shared__ __align__(16) float rk[C], rq[C], bs[4][C];
    __shared__ int badrow[C], badtok[4];

    const int kh = (int)blockIdx.y;
    const SeqTile tile = seq_tile(p.seq, C, (int)blockIdx.x);
    const int64_t t0 = (int64_t)tile.index * C;
    if (t0 >= tile.len)
        return;
    const int rows = (int)(tile.len - t0 < C ? tile.len - t0 : C);
    const int64_t first = tile.begin + t0;
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, r = lane & 15;

    // Rows of K and Q, zeros past the sequence's end and past Dk. All loads
    // go out before the first is used.
    if (tid < C)
        badrow[tid] = 0;
    lds_barrier();
    constexpr int PIECES = C * D / E / NT;
    u32x4 kv[PIECES], qv[PIECES];
    if (a.vec) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int row = (i * NT + tid) / (D / E), c = (i * NT + tid) % (D / E) * E;
            const int64_t at = first + min(row, rows - 1);
            const int cc = c < p.Dk ? c : 0;
            kv[i] = *reinterpret_cast<const u32x4 *>(static_cast<const T *>(p.k) + at * p.kst + kh * p.ksh + cc);
            qv[i] = *reinterpret_cast<const u32x4 *>(static_cast<const T *>(p.q) + at * p.qst + kh * p.qsh + cc);
        }
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int row = (i * NT + tid) / (D / E), c = (i * NT + tid) % (D / E) * E;
            if (row >= rows || c >= p.Dk)
                kv[i] = qv[i] = u32x4{0, 0, 0, 0};
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < PIECES; ++i) {
            const int row = (i * NT + tid) / (D / E), c = (i * NT + tid) % (D / E) * E;
            T k8[E] __attribute__((aligned(16))) = {}, q8[E] __attribute__((aligned(16))) = {};
            if (row < rows) {
                const T *kp = static_cast<const T *>(p.k) + (first + row) * p.kst + kh * p.ksh + c;
                const T *qp = static_cast<const T *>(p.q) + (first + row) * p.qst + kh * p.qsh + c;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (c + e < p.Dk) {
                        k8[e] = kp[e];
                        q8[e] = qp[e];
                    }
            }
            *reinterpret_cast<u32x4 *>(ks + row * PITCH + c) = *reinterpret_cast<const u32x4 *>(k8);
            *reinterpret_cast<u32x4 *>(qs + row * PITCH + c) = *reinterpret_cast<const u32x4 *>(q8);
        }
        // Each thread takes its own pieces back.
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int row = (i * NT + tid) / (D / E), c = (i * NT + tid) % (D / E) * E;
            kv[i] = *reinterpret_cast<const u32x4 *>(ks + row * PITCH + c);
            qv[i] = *reinterpret_cast<const u32x4 *>(qs + row * PITCH + c);
        }
    }
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int row = (i * NT + tid) / (D / E), c = (i * NT + tid) % (D / E) * E;
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            bad |= (!F32 && (kv[i][e] & 0x7f80u) == 0x7f80u) || (kv[i][e] & 0x7f800000u) == 0x7f800000u;
        if (bad) {
            kv[i] = u32x4{0, 0, 0, 0};
            badrow[row] = 1;
        }
        *reinterpret_cast<u32x4 *>(ks + row * PITCH + c) = kv[i];
        *reinterpret_cast<u32x4 *>(qs + row * PITCH + c) = qv[i];
    }
    lds_barrier();
    {   // four threads a row
        const int row = tid >> 2;
        float sk = 0.f, sq = 0.f;
#pragma unroll
        for (int c = E * (tid & 3); c < D; c += 4 * E) {
            const u32x4 x = *reinterpret_cast<const u32x4 *>(ks + row * PITCH + c);
            const u32x4 y = *reinterpret_cast<const u32x4 *>(qs + row * PITCH + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (F32) {
                    sk = fmaf(__uint_as_float(x[e]), __uint_as_float(x[e]), sk);
                    sq = fmaf(__uint_as_float(y[e]), __uint_as_float(y[e]), sq);
                } else {
                    const float x0 = __uint_as_float(x[e] << 16), x1 = __uint_as_float(x[e] & 0xffff0000u);
                    const float y0 = __uint_as_float(y[e] << 16), y1 = __uint_as_float(y[e] & 0xffff0000u);
                    sk = fmaf(x1, x1, fmaf(x0, x0, sk));
                    sq = fmaf(y1, y1, fmaf(y0, y0, sq));
                }
            }
        }
        sk += __shfl_xor(sk, 1);
        sk += __shfl_xor(sk, 2);
        sq += __shfl_xor(sq, 1);
        sq += __shfl_xor(sq, 2);
        if ((tid & 3) == 0) {
            rk[row] = p.normalize ? 1.f / sqrtf(sk + UNIT_EPS) : 1.f;
            rq[row] = (p.normalize ? 1.f / sqrtf(sq + UNIT_EPS) : 1.f) * p.scale;
        }
    }

    // K and Q as fragments.
    uint8_t *key = a.keys + ((int64_t)blockIdx.x * p.Hk + kh) * W::KEY;
    if constexpr (F32) {
        if (blockIdx.z == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const int at = (16 * i + r) * PITCH + 16 * (DT * w + d) + 4 * g;
                    f32x4 f;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        f[e] = ks[(16 * i + 4 * g + e) * PITCH + 16 * (DT * w + d) + r];
                    reinterpret_cast<f32x4 *>(key + ((4 * w + i) * DT + d) * FRAG)[lane] =
                        *reinterpret_cast<const f32x4 *>(ks + at);
                    reinterpret_cast<f32x4 *>(key + W::Q + ((4 * i + w) * DT + d) * FRAG)[lane] =
                        *reinterpret_cast<const f32x4 *>(qs + at);
                    reinterpret_cast<f32x4 *>(key + W::KT + ((DT * w + d) * 4 + i) * FRAG)[lane] = f;
                }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {       // wave w writes what wave w of the second kernel reads
            const int at = token_of(i, r) * PITCH + (DT == 2 ? 32 * w + 8 * g : 16 * w + 4 * g);
            u32x4 kf = {0, 0, 0, 0}, qf = {0, 0, 0, 0};
            if constexpr (DT == 2) {
                kf = *reinterpret_cast<const u32x4 *>(ks + at);
                qf = *reinterpret_cast<const u32x4 *>(qs + at);
            } else {
                const u32x2 k2 = *reinterpret_cast<const u32x2 *>(ks + at), q2 = *reinterpret_cast<const u32x2 *>(qs + at);
                kf[0] = k2[0], kf[1] = k2[1];
                qf[0] = q2[0], qf[1] = q2[1];
            }
            if (blockIdx.z == 0) {
                reinterpret_cast<u32x4 *>(key + (4 * w + i) * FRAG)[lane] = kf;
                reinterpret_cast<u32x4 *>(key + W::Q + (4 * i + w) * FRAG)[lane] = qf;
            }
        }
    }

    // Row tile w of K K^T and Q K^T (rows in token order here).
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        kk[j] = qk[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (F32) {
#pragma unroll 2
        for (int s = 0; s < D / 16; ++s) {
            const int c = 16 * s + 4 * g;
            const f32x4 ka = *reinterpret_cast<const f32x4 *>(ks + (16 * w + r) * PITCH + c);
            const f32x4 qa = *reinterpret_cast<const f32x4 *>(qs + (16 * w + r) * PITCH + c);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= w) {
                    const f32x4 kb = *reinterpret_cast<const f32x4 *>(ks + (16 * j + r) * PITCH + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        kk[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(ka[e], kb[e], kk[j], 0, 0, 0);
                        qk[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(qa[e], kb[e], qk[j], 0, 0, 0);
                    }
                }
        }
    } else {
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
            const int c = 32 * s + 8 * g;
            const bf16x8 ka = *reinterpret_cast<const bf16x8 *>(ks + (16 * w + r) * PITCH + c);
            const bf16x8 qa = *reinterpret_cast<const bf16x8 *>(qs + (16 * w + r) * PITCH + c);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= w) {
                    const bf16x8 kb = *reinterpret_cast<const bf16x8 *>(ks + (16 * j + r) * PITCH + c);
                    kk[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ka, kb, kk[j], 0, 0, 0);
                    qk[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qa, kb, qk[j], 0, 0, 0);
                }
        }
    }

    lds_barrier();
    for (int i = tid; i < C * MP / 4; i += NT)
        reinterpret_cast<f32x4 *>(m)[i] = reinterpret_cast<f32x4 *>(pm)[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int group = p.Hv / p.Hk, h0 = (int)blockIdx.z * a.heads, heads = min(a.heads, group - h0);
    for (int hi = 0; hi < heads; ++hi) {
        const int h = kh * group + h0 + hi, hs = hi & 3;
        if (hs == 0) {
            // Sums of the gates of the next four heads, a wave each, in 64
            // bits; a total gate counts as exp(-10000) = 0.
            lds_barrier();
            if (hi + w < heads) {
                float gate = 0.f, beta = 0.f;
                if (lane < rows) {
                    gate = p.g[(first + lane) * p.Hv + h + w];
                    beta = p.beta[(first + lane) * p.Hv + h + w];
                }
                const bool bad = !(gate < INFINITY) || !(fabsf(beta) < INFINITY) || badrow[lane];
                const uint64_t bads = __ballot(bad);
                if (bad) {
                    gate = gate < INFINITY ? gate : 0.f;
                    beta = 0.f;
                }
                double G = (double)fmaxf(gate, -1e4f);
#pragma unroll
                for (int d = 1; d < 64; d <<= 1) {
                    const double o = __shfl_up(G, d);
                    if (lane >= d)
                        G += o;
                }
                gs[w][lane] = G;
                bs[w][lane] = beta;
                if (lane == 0)
                    badtok[w] = bads ? __builtin_ctzll(bads) : NEVER;
            }
        }
        lds_barrier();
        {
            const int row0 = 16 * w + 4 * g;
            double gr[4];
            float ar[4], pr[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                gr[e] = gs[hs][row0 + e];
                ar[e] = bs[hs][row0 + e] * rk[row0 + e];
                pr[e] = rq[row0 + e];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= w) {
                    const int col = 16 * j + r;
                    const double gc = gs[hs][col];
                    const float rc = rk[col];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float d = __expf((float)(gr[e] - gc)) * rc;
                        m[(row0 + e) * MP + col] = row0 + e > col ? ar[e] * d * kk[j][e] : 0.f;
                        pm[(row0 + e) * MP + col] = row0 + e >= col ? pr[e] * d * qk[j][e] : 0.f;
                    }
                }
        }
        lds_barrier();
        // (1 + A)^-1: the 16x16 blocks on the diagonal by substitution, lane c
        // a column, then blocks twice as large from
        //   [[X, 0], [A, Y]]^-1 = [[X^-1, 0], [-Y^-1 A X^-1, Y^-1]].
        if (lane < 16) {
            float col[16];
            float *blk = m + 16 * w * MP + 16 * w;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float x = i == lane ? 1.f : 0.f;
#pragma unroll
                for (int j = 0; j < i; ++j)
                    x = fmaf(-blk[i * MP + j], col[j], x);
                col[i] = x;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
                blk[i * MP + lane] = col[i];
        }
        lds_barrier();
        // A X^-1's rows that overflowed would meet the zeros of Y^-1 in earlier tokens' rows. (Elsewhere rows of A and T
        // that are not finite stay in theirs, and U shows them.)
        auto finite = [&](f32x4 &t, int token) __attribute__((always_inline)) {
            const float zero = fmaf(t[0], 0.f, fmaf(t[1], 0.f, fmaf(t[2], 0.f, t[3] * 0.f)));
            if (__any(zero != 0.f))
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!(fabsf(t[e]) < INFINITY)) {
                        atomicMin(&badtok[hs], token + e);
                        t[e] = 0.f;
                    }
        };
        if (w < 2) {
            const int i = 2 * w + 1, j = 2 * w;
            f32x4 t = {0.f, 0.f, 0.f, 0.f}, o = t;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                t = __builtin_amdgcn_mfma_f32_16x16x4f32(m[(16 * i + r) * MP + 16 * j + 4 * e + g],
                                                         m[(16 * j + 4 * e + g) * MP + 16 * j + r], t, 0, 0, 0);
            finite(t, 16 * i + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o = __builtin_amdgcn_mfma_f32_16x16x4f32(m[(16 * i + r) * MP + 16 * i + 4 * g + e], t[e], o, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                m[(16 * i + 4 * g + e) * MP + 16 * j + r] = -o[e];
        }
        lds_barrier();
        {
            const int i = 2 + (w >> 1), j = w & 1;
            f32x4 t = {0.f, 0.f, 0.f, 0.f}, o = t;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (k >= j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        t = __builtin_amdgcn_mfma_f32_16x16x4f32(m[(16 * i + r) * MP + 16 * k + 4 * e + g],
                                                                 m[(16 * k + 4 * e + g) * MP + 16 * j + r], t, 0, 0, 0);
            finite(t, 16 * i + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                z(w)[(4 * g + e) * MP + r] = t[e];
            lds_barrier();
#pragma unroll
            for (int k = 2; k < 4; ++k)
                if (k <= i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o = __builtin_amdgcn_mfma_f32_16x16x4f32(m[(16 * i + r) * MP + 16 * k + 4 * e + g],
                                                                 z(2 * (k - 2) + j)[(4 * e + g) * MP + r], o, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                m[(16 * i + 4 * g + e) * MP + 16 * j + r] = -o[e];
        }
        lds_barrier();

        uint8_t *val = a.vals + ((int64_t)blockIdx.x * p.Hv + h) * W::VAL;
        if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= w) {
                    const int col = 16 * j + 4 * g, f = w * (w + 1) / 2 + j;
                    reinterpret_cast<f32x4 *>(val + f * FRAG)[lane] =
                        *reinterpret_cast<const f32x4 *>(m + (16 * w + r) * MP + col) *
                        *reinterpret_cast<const f32x4 *>(bs[hs] + col);
                    reinterpret_cast<f32x4 *>(val + W::P + f * FRAG)[lane] =
                        *reinterpret_cast<const f32x4 *>(pm + (16 * w + r) * MP + col);
                }
        } else {
            const int row = token_of(w, r);
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (2 * s <= w) {
                    bf16x8 t3[3];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int col = 32 * s + 8 * g + e;
                        float t = m[row * MP + col] * bs[hs][col];
                        t3[0][e] = part_of(t);
                        t3[1][e] = part_of(t);
                        t3[2][e] = part_of(t);
                    }
                    const int f = low_frag(w, s);
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        reinterpret_cast<bf16x8 *>(val + (3 * f + i) * FRAG)[lane] = t3[i];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        reinterpret_cast<f32x4 *>(val + W::P + (2 * f + i) * FRAG)[lane] =
                            *reinterpret_cast<const f32x4 *>(pm + row * MP + 32 * s + 8 * g + 4 * i);
                }
        }
        if (w == 0) {
            const double G = gs[hs][lane], last = gs[hs][C - 1];
            const float e = __expf((float)G);
            reinterpret_cast<float *>(val + W::UPK)[lane] = e * rk[lane];
            reinterpret_cast<float *>(val + W::UPQ)[lane] = e * rq[lane];
            reinterpret_cast<float *>(val + W::TAIL)[lane] = __expf((float)(last - G)) * rk[lane];
            if (lane == 0) {
                reinterpret_cast<float *>(val + W::HEAD)[0] = __expf((float)last);
                reinterpret_cast<int *>(val + W::HEAD)[1] = badtok[hs];
            }
        }
    }
}

// x as bf16 parts, the nearest bf16 of what the parts before left. Two values
// a conversion; a part's value is its bits in the upper half of a float.
template <int N>
__device__ __forceinline__ void split(const f32x4 &x, bf16x4 (&part)[N])
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    f32x4 left = x;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t lo = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{left[0], left[1]}), bf16x2));
        const uint32_t hi = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{left[2], left[3]}), bf16x2));
        part[i] = __builtin_bit_cast(bf16x4, (u32x2{lo, hi}));
        if (i + 1 < N) {
            left[0] -= __uint_as_float(lo << 16);
            left[1] -= __uint_as_float(lo & 0xffff0000u);
            left[2] -= __uint_as_float(hi << 16);
            left[3] -= __uint_as_float(hi & 0xffff0000u);
        }
    }
}

// Two tiles of U, four tokens of a column each from `token` and token + apart
// on. One that is not finite (it has overflowed) is noted in *bad and set to
// zero, since P's zeros would carry it to earlier tokens.
__device__ __forceinline__ void finite_u(f32x4 &a, f32x4 &b, int *bad, int token, int apart)
{
    float zero = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        zero = fmaf(a[e], 0.f, fmaf(b[e], 0.f, zero));
    if (!__any(zero != 0.f))
        return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (!(fabsf(a[e]) < INFINITY)) {
            atomicMin(bad, token + e);
            a[e] = 0.f;
        }
        if (!(fabsf(b[e]) < INFINITY)) {
            atomicMin(bad, token + apart + e);
            b[e] = 0.f;
        }
    }
}

__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// Values of four lanes transposed: of each 16 lanes, lane i gets value i % 4 of
// the places of lanes i / 4, 4 + i / 4, 8 + i / 4 and 12 + i / 4.
__device__ __forceinline__ bf16x4 transposed(const bf16x4 *place)
{
    typedef short i16x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                          (__attribute__((address_space(3))) i16x4 *)(place)));
}

// Waves 0 to 3 carry S, waves 4 to 7 make the outputs. Three exchanges
// through LDS a chunk, each ended by a barrier that all eight waves meet:
//   chain wave w: its rows' share of K S; its rows of S in three parts -> xp; ssh
//   chain wave w: token tile w of Y in three parts                    -> ysh
//   chain wave w: token tile w of U, for S' in three parts and for O  -> ush; uo
// then chain wave w updates its rows of S. Output wave w takes Q S between the
// first two barriers, stores the chunk before and splits its rows of P between
// the second and the third, and after it brings V and the row factors of the
// next chunk and adds P U. The time of a chunk is the chain's latencies, not
// its arithmetic, so whatever is not the chain is left to the output waves, and
// every operand is loaded right after its last use, a chunk ahead. (16384
// tokens, this kernel: 758 us with four waves that did all, 467 with the split,
// 430 with K^T transposed out of LDS instead of loaded beside K; that with two
// parts of S, U and P for the outputs, 2^-17, and 465 with all three. P split
// only where it is used, 16384 tokens are no slower, and 16 heads of 64 x 64 4 %.)
// VEC: v's rows of 16 columns are two 16-byte pieces and o's take 8-byte
// stores (a host rule; as a branch inside, it made the compiler wait for
// every load at its end).
template <int DT, bool VEC>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(4))) void delta_chunks_kernel(ChunkArgs a)
{
    using W = Space<DT, false>;
    const DeltaProblem &p = a.p;
    __shared__ f32x4 xp[4][4][64], uo[4][64];
    __shared__ bf16x8 ssh[3][4][64];
    __shared__ bf16x4 ysh[3][4][64], ush[3][4][64];
    __shared__ bf16x4 ksh[4][4][DT][64];            // chain wave w's K, for its transposed reads
    __shared__ f32x4 vsh[4][64], factors[4][2][4];  // factors: r exp G, then r exp(G_63 - G)
    __shared__ u32x4 vrows[4][32];                  // V as it lies in memory: 16 tokens of 32 bytes
    __shared__ __align__(16) int badcol[16];

    // Workgroup i runs on XCD i % 8. The slices of one head go to one XCD,
    // where they meet in its L2; the heads of a sequence, as long as each
    // other, go round the XCDs.
    const int at = (int)blockIdx.x >> 3;
    const int slice = at % a.slices, nh = at / a.slices * 8 + ((int)blockIdx.x & 7);
    if (nh >= p.seq.num_seqs * p.Hv)
        return;
    const int n = nh / p.Hv, h = nh % p.Hv, kh = h / (p.Hv / p.Hk);
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int w8 = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    // Token tiles 2 and 3 have twice the work of 0 and 1, in both roles: the
    // output wave of a SIMD takes the other half's tile.
    const int w = w8 < 4 ? w8 : 7 - w8;
    const int64_t begin = seq_begin(p.seq, n);
    const int64_t end = seq_begin(p.seq, n + 1);
    const int len = end > begin ? (int)(end - begin) : 0;
    const int chunks = (len + C - 1) / C;
    const int64_t number = begin / C + n;
    const int slot = p.state_in || p.state_out ? seq_slot(p.seq, n) : -1;
    const int col0 = slice * 16;
    const int tok4 = 32 * (w >> 1) + 8 * g + 4 * (w & 1);      // first of the lane's four tokens of tile w
    const int tokr = token_of(w, r);
    const uint8_t *key0 = a.keys + (number * p.Hk + kh) * W::KEY;
    const uint8_t *val0 = a.vals + (number * p.Hv + h) * W::VAL;
    const int64_t key_step = (int64_t)p.Hk * W::KEY, val_step = (int64_t)p.Hv * W::VAL;
    // Fragment i from a base that is the same for all lanes: such a load needs no vector address arithmetic while
    // i * FRAG fits the instruction's offset (-4096 .. 4095 bytes).
    const uint32_t lane16 = 16 * lane;
    auto frag = [&](const uint8_t *base, int i) __attribute__((always_inline)) {
        return *reinterpret_cast<const bf16x8 *>(base + lane16 + i * FRAG);
    };

    if (threadIdx.x < 16)
        badcol[threadIdx.x] = NEVER;
    __syncthreads();

    if (w8 >= 4) {
        // ---- Output wave w: token tile w of O, as rows of columns 4g .. 4g + 3, token r.
        bf16x8 qf[4];
        f32x4 pf[2][2];
        float upq = 0.f;
        int bad_here = NEVER, badall = NEVER;
        auto load_q = [&](int c) __attribute__((always_inline)) {
            const uint8_t *key = key0 + c * key_step + W::Q + 4 * w * FRAG;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                qf[i] = frag(key, i);
        };
        auto load_p = [&](int c) __attribute__((always_inline)) {
            const uint8_t *pv = val0 + c * val_step + W::P + 2 * low_frag(w, 0) * FRAG;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    pf[s][i] = __builtin_bit_cast(f32x4, frag(pv, 2 * s + i));  // s = 1 of waves 0 and 1: the next wave's, not used
        };
        auto load_rows = [&](int c) __attribute__((always_inline)) {
            const uint8_t *val = val0 + c * val_step;
            upq = reinterpret_cast<const float *>(val + W::UPQ)[tokr];
            bad_here = reinterpret_cast<const int *>(val + W::HEAD)[1];
        };
        // V and the row factors of chain wave w's tokens, on to it through LDS.
        uint16_t v[4];
        u32x4 vpiece;
        f32x4 factor;
        const uint16_t *vh = static_cast<const uint16_t *>(p.v) + begin * p.vst + h * p.vsh;
        const int64_t voff = tok4 * p.vst;      // of the lane's first token within a chunk
        const int vcol = min(col0 + r, p.Dv - 1);   // columns past the end read the last one's; nothing is stored of them
        auto load_v = [&](int c) __attribute__((always_inline)) {
            factor = *reinterpret_cast<const f32x4 *>(val0 + c * val_step + (r < 8 ? W::UPK : W::TAIL) + 4 * tok4);
            const uint16_t *vc = vh + (int64_t)c * C * p.vst;
            // Tokens past the end read the last one's: T's columns are zero for
            // them. (No branch: the compiler would wait for the loads at its end.)
            const int last = len - 1 - c * C;
            if constexpr (VEC) {        // half a token's 32 bytes a lane
                const uint16_t *row = vc + min(token_of(w, (lane >> 1) & 15), last) * p.vst + col0 + 8 * (lane & 1);
                vpiece = *reinterpret_cast<const u32x4 *>(row);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int64_t off = tok4 + e <= last ? voff : (last - e) * p.vst;
                    v[e] = (vc + e * p.vst + off)[vcol];
                }
            }
        };
        auto give_v = [&]() __attribute__((always_inline)) {
            if constexpr (VEC) {
                if (lane < 32)
                    vrows[w][lane] = vpiece;
                const uint16_t *rows = reinterpret_cast<const uint16_t *>(vrows[w]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = rows[16 * (4 * g + e) + r];
            }
            vsh[w][lane] = f32x4{bf16_to_f32(v[0]), bf16_to_f32(v[1]), bf16_to_f32(v[2]), bf16_to_f32(v[3])};
            if ((r & 7) == 0)
                factors[w][r >> 3][g] = factor;
        };
        if (chunks > 0) {
            load_v(0);
            give_v();
            load_v(min(1, chunks - 1));
            load_q(0);
            load_p(0);
            load_rows(0);
        }
        uint16_t *oh = static_cast<uint16_t *>(p.o) + (begin + tokr) * p.ost + h * p.osh + col0 + 4 * g;
        f32x4 o;
        // P in parts, before the phase that needs them.
        bf16x8 pp[2][3];
        auto split_p = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (2 * s <= w) {
                    bf16x4 lo[3], hi[3];
                    split<3>(pf[s][0], lo);
                    split<3>(pf[s][1], hi);
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        pp[s][i] = join(lo[i], hi[i]);
                }
        };
        // The second term of chunk c's outputs.
        auto add_pu = [&](int c) __attribute__((always_inline)) {
            // Nothing that looks at these two may move up to their load, a
            // phase earlier: it would wait there.
            asm volatile("" : "+v"(bad_here), "+v"(upq));
            if (badall == NEVER && bad_here != NEVER)
                badall = c * C + bad_here;
            o *= upq;
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (2 * s <= w) {
                    f32x4 ua = uo[2 * s][lane], ub = uo[2 * s + 1][lane];
                    finite_u(ua, ub, &badcol[r], c * C + 32 * s + 8 * g, 4);
                    bf16x4 lo[3], hi[3];
                    bf16x8 u[3];
                    split<3>(ua, lo);
                    split<3>(ub, hi);
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        u[i] = join(lo[i], hi[i]);
#pragma unroll
                    for (int k = 2; k >= 0; --k)
#pragma unroll
                        for (int i = 0; i <= k; ++i)
                            o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u[k - i], pp[s][i], o, 0, 0, 0);
                }
        };
        auto store = [&](int c) __attribute__((always_inline)) {
            const int t = c * C + tokr;
            const i32x4 bc = *reinterpret_cast<const i32x4 *>(badcol + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = t >= min(badall, bc[e]) ? NAN : o[e];
            if (t < len) {
                if constexpr (VEC) {
                    *reinterpret_cast<bf16x4 *>(oh) = __builtin_convertvector(o, bf16x4);
                } else {
                    const int left = p.Dv - (col0 + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < left)
                            oh[e] = f32_to_bf16_rne(o[e]);
                }
            }
            oh += C * p.ost;
        };
        for (int c = 0; c < chunks; ++c) {
            lds_barrier();
            // S^T Q^T, every wave's rows of S.
            f32x4 q = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 2; j >= 0; --j)
                    q = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ssh[j][i][lane], qf[i], q, 0, 0, 0);
            load_q(min(c + 1, chunks - 1));
            lds_barrier();
            if (c > 0)
                store(c - 1);
            o = q;
            split_p();
            load_p(min(c + 1, chunks - 1));
            lds_barrier();
            // For the next chunk: the chain reads them between the next two
            // barriers, and took its last look at this chunk's before the one above.
            give_v();
            load_v(min(c + 2, chunks - 1));
            add_pu(c);
            load_rows(min(c + 1, chunks - 1));
        }
        if (chunks > 0)
            store(chunks - 1);
        return;
    }

    // ---- Chain wave w: its rows of S, as results leave the matrix cores
    // (row dk_of(d) + e, column r of each 16).
    const int64_t sat = ((int64_t)slot * p.Hv + h) * p.Dk * p.Dv;
    auto dk_of = [&](int d) { return DT == 2 ? 32 * w + 8 * g + 4 * d : 16 * w + 4 * g; };
    f32x4 S[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // All loads at once: what is past the state reads its last row and column.
            const int dk = dk_of(d) + e, col = col0 + r;
            float v = 0.f;
            if (p.state_in && slot >= 0)
                v = p.state_in[sat + (int64_t)min(dk, p.Dk - 1) * p.Dv + min(col, p.Dv - 1)];
            S[d][e] = dk < p.Dk && col < p.Dv ? v : 0.f;
        }

    bf16x8 kf[4], tf[2][3];
    u32x2 head = {0, 0};
    bool bad_any = false;       // some token of a chunk so far is not finite
    auto load_k = [&](int c) __attribute__((always_inline)) {
        const uint8_t *key = key0 + c * key_step + 4 * w * FRAG;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            kf[i] = frag(key, i);
    };
    auto load_t = [&](int c) __attribute__((always_inline)) {
        const uint8_t *val = val0 + c * val_step + (3 * low_frag(w, 0) + 2) * FRAG;
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (2 * s <= w)
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    tf[s][i] = frag(val, 3 * s + i - 2);
    };
    auto load_head = [&](int c) __attribute__((always_inline)) {
        // (A scalar load would be waited for at the next barrier, which waits
        // for LDS traffic on the same counter.)
        head = *reinterpret_cast<const u32x2 *>(val0 + c * val_step + W::HEAD);
    };
    if (chunks > 0) {
        load_k(0);
        load_t(0);
        load_head(0);
    }
    __builtin_amdgcn_s_setprio(3);      // before the output wave of the same SIMD
    for (int c = 0; c < chunks; ++c) {
        const int next = min(c + 1, chunks - 1);
        // K S, wave w's rows of S only.
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ksh[w][i][0][4 * r + g] = __builtin_shufflevector(kf[i], kf[i], 0, 1, 2, 3);
            if constexpr (DT == 2)
                ksh[w][i][DT - 1][4 * r + g] = __builtin_shufflevector(kf[i], kf[i], 4, 5, 6, 7);
        }
        bf16x4 lo[3], hi[3] = {};
        split<3>(S[0], lo);
        if constexpr (DT == 2)
            split<3>(S[DT - 1], hi);
        f32x4 acc[4] = {};
#pragma unroll
        for (int j = 2; j >= 0; --j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[i], join(lo[j], hi[j]), acc[i], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            xp[w][i][lane] = acc[i];
#pragma unroll
        for (int j = 0; j < 3; ++j)
            ssh[j][w][lane] = join(lo[j], hi[j]);
        load_k(next);
        lds_barrier();
        // Token tile w of Y = V - diag(r exp G) K S.
        f32x4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = xp[i][w][lane];
        const f32x4 v = vsh[w][lane], up = factors[w][0][g];
        __builtin_amdgcn_sched_barrier(0);      // all reads before the first sum
        f32x4 y = v - up * ((x[0] + x[1]) + (x[2] + x[3]));
        float zero = 0.f;                       // NaN if anything of y is not finite
#pragma unroll
        for (int e = 0; e < 4; ++e)
            zero = fmaf(y[e], 0.f, zero);
        if (__any(zero != 0.f))
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!(fabsf(y[e]) < INFINITY)) {
                    atomicMin(&badcol[r], c * C + tok4 + e);
                    y[e] = 0.f;
                }
        bf16x4 part[3];
        split<3>(y, part);
#pragma unroll
        for (int i = 0; i < 3; ++i)
            ysh[i][w][lane] = part[i];
        lds_barrier();
        // Token tile w of U = T Y.
        const f32x4 tail = factors[w][1][g];
        f32x4 u = {0.f, 0.f, 0.f, 0.f};
        bf16x8 yf[2][3];
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (2 * s <= w)
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    yf[s][i] = join(ysh[i][2 * s][lane], ysh[i][2 * s + 1][lane]);
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (2 * s <= w)
#pragma unroll
                for (int k = 2; k >= 0; --k)
#pragma unroll
                    for (int i = 0; i <= k; ++i)
                        u = __builtin_amdgcn_mfma_f32_16x16x32_bf16(tf[s][i], yf[s][k - i], u, 0, 0, 0);
        uo[w][lane] = u;
        bf16x4 us[3];
        split<3>(u * tail, us);
#pragma unroll
        for (int i = 0; i < 3; ++i)
            ush[i][w][lane] = us[i];
        // K^T for the last phase: lane (g, r) gets values r % 4 of lanes
        // (r / 4, 4g + e), which lie together.
        bf16x8 ktf[DT][2];
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                ktf[d][s] = join(transposed(ksh[w][2 * s][d] + lane), transposed(ksh[w][2 * s + 1][d] + lane));
        load_t(next);
        lds_barrier();
        // S'.
        bad_any |= (int)head[1] != NEVER;
#pragma unroll
        for (int d = 0; d < DT; ++d)
            S[d] *= __uint_as_float(head[0]);
#pragma unroll
        for (int i = 2; i >= 0; --i)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const bf16x8 u = join(ush[i][2 * s][lane], ush[i][2 * s + 1][lane]);
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    S[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ktf[d][s], u, S[d], 0, 0, 0);
            }
        load_head(next);
    }
    if (!p.state_out || slot < 0)
        return;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int dk = dk_of(d) + e, col = col0 + r;
            const bool bad = bad_any || badcol[r] != NEVER || (chunks > 0 && !(fabsf(S[d][e]) < INFINITY));
            if (dk < p.Dk && col < p.Dv)
                p.state_out[sat + (int64_t)dk * p.Dv + col] = bad ? NAN : S[d][e];
        }
}

// The same in fp32 with fp32 matrix instructions (16x16x4). A result's four
// rows a lane are the next product's operand as they lie, value e for step e,
// so nothing is split and tokens keep their order; the waves, barriers and the
// order of loads are those of the kernel above. 2047 tokens, 16 heads of 128 x
// 128: 118 us with the preparation, token by token 1500. The instructions are
// half of a chunk's 2.8 us. 128 registers (two spilled) for two workgroups a
// compute unit: 8 sequences of 256 tokens, 32 heads, 167 -> 150 us.
template <int DT>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(4))) void delta_chunks_f32_kernel(ChunkArgs a)
{
    using W = Space<DT, true>;
    const DeltaProblem &p = a.p;
    __shared__ f32x4 xp[4][4][64], ssh[4][DT][64], ysh[4][64], ush[4][64], uo[4][64], vsh[4][64];
    __shared__ f32x4 factors[4][2][4];
    __shared__ int badcol[16];

    const int at = (int)blockIdx.x >> 3;
    const int slice = at % a.slices, nh = at / a.slices * 8 + ((int)blockIdx.x & 7);
    if (nh >= p.seq.num_seqs * p.Hv)
        return;
    const int n = nh / p.Hv, h = nh % p.Hv, kh = h / (p.Hv / p.Hk);
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int w8 = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int w = w8 < 4 ? w8 : 7 - w8;
    const int64_t begin = seq_begin(p.seq, n);
    const int64_t end = seq_begin(p.seq, n + 1);
    const int len = end > begin ? (int)(end - begin) : 0;
    const int chunks = (len + C - 1) / C;
    const int64_t number = begin / C + n;
    const int slot = p.state_in || p.state_out ? seq_slot(p.seq, n) : -1;
    const int col = slice * 16 + r;
    const int tok4 = 16 * w + 4 * g;
    const uint8_t *key0 = a.keys + (number * p.Hk + kh) * W::KEY;
    const uint8_t *val0 = a.vals + (number * p.Hv + h) * W::VAL;
    const int64_t key_step = (int64_t)p.Hk * W::KEY, val_step = (int64_t)p.Hv * W::VAL;
    const uint32_t lane16 = 16 * lane;
    auto frag = [&](const uint8_t *base, int i) __attribute__((always_inline)) {
        return *reinterpret_cast<const f32x4 *>(base + lane16 + i * FRAG);
    };
    auto mac = [](const f32x4 &x, const f32x4 &y, f32x4 sum) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sum = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], sum, 0, 0, 0);
        return sum;
    };
    const int low = w * (w + 1) / 2;        // first fragment of row tile w of T and P

    if (threadIdx.x < 16)
        badcol[threadIdx.x] = NEVER;
    __syncthreads();

    if (w8 >= 4) {
        f32x4 qf[4 * DT], pf[4], upq = {}, o;
        int bad_here = NEVER, badall = NEVER;
        auto load_q = [&](int c) __attribute__((always_inline)) {
            const uint8_t *key = key0 + c * key_step + W::Q + 4 * DT * w * FRAG;
#pragma unroll
            for (int i = 0; i < 4 * DT; ++i)
                qf[i] = frag(key, i);
        };
        auto load_p = [&](int c) __attribute__((always_inline)) {
            const uint8_t *val = val0 + c * val_step, *pv = val + W::P + low * FRAG;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                pf[j] = frag(pv, min(j, w));
            upq = *reinterpret_cast<const f32x4 *>(val + W::UPQ + 4 * tok4);
            bad_here = reinterpret_cast<const int *>(val + W::HEAD)[1];
        };
        float v[4];
        f32x4 factor;
        const float *vh = static_cast<const float *>(p.v) + begin * p.vst + h * p.vsh + min(col, p.Dv - 1);
        auto load_v = [&](int c) __attribute__((always_inline)) {
            factor = *reinterpret_cast<const f32x4 *>(val0 + c * val_step + (r < 8 ? W::UPK : W::TAIL) + 4 * tok4);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = vh[min(c * C + tok4 + e, len - 1) * p.vst];
        };
        auto give_v = [&]() __attribute__((always_inline)) {
            vsh[w][lane] = f32x4{v[0], v[1], v[2], v[3]};
            if ((r & 7) == 0)
                factors[w][r >> 3][g] = factor;
        };
        if (chunks > 0) {
            load_v(0);
            give_v();
            load_v(min(1, chunks - 1));
            load_q(0);
            load_p(0);
        }
        float *oh = static_cast<float *>(p.o) + (begin + tok4) * p.ost + h * p.osh + col;
        auto add_pu = [&](int c) __attribute__((always_inline)) {
            asm volatile("" : "+v"(bad_here));      // (not looked at before this phase, see above)
            if (badall == NEVER && bad_here != NEVER)
                badall = c * C + bad_here;
            o *= upq;
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (2 * s <= w) {
                    f32x4 ua = uo[2 * s][lane], ub = uo[2 * s + 1][lane];
                    finite_u(ua, ub, &badcol[r], c * C + 32 * s + 4 * g, 16);
                    o = mac(pf[2 * s], ua, o);
                    if (2 * s < w)
                        o = mac(pf[2 * s + 1], ub, o);
                }
        };
        auto store = [&](int c) __attribute__((always_inline)) {
            const int bad = min(badall, badcol[r]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = c * C + tok4 + e;
                if (t < len && col < p.Dv)
                    oh[e * p.ost] = t >= bad ? NAN : o[e];
            }
            oh += C * p.ost;
        };
        for (int c = 0; c < chunks; ++c) {
            lds_barrier();
            f32x4 q = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    q = mac(qf[DT * i + d], ssh[i][d][lane], q);
            load_q(min(c + 1, chunks - 1));
            lds_barrier();
            if (c > 0)
                store(c - 1);
            o = q;
            lds_barrier();
            give_v();
            load_v(min(c + 2, chunks - 1));
            add_pu(c);
            load_p(min(c + 1, chunks - 1));
        }
        if (chunks > 0)
            store(chunks - 1);
        return;
    }

    const int64_t sat = ((int64_t)slot * p.Hv + h) * p.Dk * p.Dv;
    auto dk_of = [&](int d) { return 16 * (DT * w + d) + 4 * g; };
    f32x4 S[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int dk = dk_of(d) + e;
            float v = 0.f;
            if (p.state_in && slot >= 0)
                v = p.state_in[sat + (int64_t)min(dk, p.Dk - 1) * p.Dv + min(col, p.Dv - 1)];
            S[d][e] = dk < p.Dk && col < p.Dv ? v : 0.f;
        }

    f32x4 kf[4][DT], ktf[DT][4], tf[4];
    u32x2 head = {0, 0};
    bool bad_any = false;
    auto load_k = [&](int c) __attribute__((always_inline)) {
        const uint8_t *key = key0 + c * key_step + 4 * DT * w * FRAG;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int d = 0; d < DT; ++d)
                kf[i][d] = frag(key, i * DT + d);
    };
    auto load_t = [&](int c) __attribute__((always_inline)) {
        const uint8_t *val = val0 + c * val_step + low * FRAG;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            tf[j] = frag(val, min(j, w));
    };
    auto load_kt = [&](int c) __attribute__((always_inline)) {
        const uint8_t *key = key0 + c * key_step + W::KT + 4 * DT * w * FRAG;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                ktf[d][j] = frag(key, 4 * d + j);
        head = *reinterpret_cast<const u32x2 *>(val0 + c * val_step + W::HEAD);
    };
    if (chunks > 0) {
        load_k(0);
        load_t(0);
        load_kt(0);
    }
    __builtin_amdgcn_s_setprio(3);
    for (int c = 0; c < chunks; ++c) {
        const int next = min(c + 1, chunks - 1);
#pragma unroll
        for (int d = 0; d < DT; ++d)
            ssh[w][d][lane] = S[d];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int d = 0; d < DT; ++d)
                acc = mac(kf[i][d], S[d], acc);
            xp[w][i][lane] = acc;
        }
        load_k(next);
        lds_barrier();
        f32x4 y = vsh[w][lane] -
                  factors[w][0][g] * ((xp[0][w][lane] + xp[1][w][lane]) + (xp[2][w][lane] + xp[3][w][lane]));
        float zero = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            zero = fmaf(y[e], 0.f, zero);
        if (__any(zero != 0.f))
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!(fabsf(y[e]) < INFINITY)) {
                    atomicMin(&badcol[r], c * C + tok4 + e);
                    y[e] = 0.f;
                }
        ysh[w][lane] = y;
        lds_barrier();
        const f32x4 tail = factors[w][1][g];
        f32x4 u = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= w)
                u = mac(tf[j], ysh[j][lane], u);
        uo[w][lane] = u;
        ush[w][lane] = u * tail;
        load_t(next);
        lds_barrier();
        bad_any |= (int)head[1] != NEVER;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            S[d] *= __uint_as_float(head[0]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                S[d] = mac(ktf[d][j], ush[j][lane], S[d]);
        }
        load_kt(next);
    }
    if (!p.state_out || slot < 0)
        return;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int dk = dk_of(d) + e;
            const bool bad = bad_any || badcol[r] != NEVER || (chunks > 0 && !(fabsf(S[d][e]) < INFINITY));
            if (dk < p.Dk && col < p.Dv)
                p.state_out[sat + (int64_t)dk * p.Dv + col] = bad ? NAN : S[d][e];
        }
}

template <int DT, bool F32>
hipError_t launch(const DeltaProblem &p, hipStream_t s)
{
    using W = Space<DT, F32>;
    ChunkArgs a = {};
    a.p = p;
    const int64_t numbers = seq_tiles(p.seq, C);
    a.keys = static_cast<uint8_t *>(p.workspace);
    a.vals = a.keys + numbers * p.Hk * W::KEY;
    a.vec = ((uintptr_t)p.q | (uintptr_t)p.k) % 16 == 0 && (p.qst | p.qsh | p.kst | p.ksh | p.Dk) % (F32 ? 4 : 8) == 0;
    const bool vec = (uintptr_t)p.v % 16 == 0 && (p.vst | p.vsh) % 8 == 0 && p.Dv % 16 == 0 && (uintptr_t)p.o % 8 == 0 &&
                     (p.ost | p.osh) % 4 == 0;
    // One value head a workgroup while the chip holds them all at once, or
    // nearly (four a compute unit): 33 chunks of 32 heads, two a key head, took
    // 85.3 us together and 84.5 apart, 65 chunks 140 and 146; 9 chunks of 16
    // heads, four a key head, 38.0 and 28.1. In fp32 (two a compute unit, and
    // more work that they would share): 17 chunks of 32 heads, two a key head,
    // 77.5 together and 83.3 apart; of 16, four a key head, 77.7 and 71.2.
    const int group = p.Hv / p.Hk;
    a.heads = numbers * p.Hv <= (F32 ? 512 : 1280) ? 1 : group;
    hipLaunchKernelGGL((delta_prepare_kernel<DT, F32>),
                       dim3((unsigned)numbers, (unsigned)p.Hk, (unsigned)((group + a.heads - 1) / a.heads)), dim3(NT), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    a.slices = (p.Dv + 15) / 16;
    const int64_t heads = ((int64_t)p.seq.num_seqs * p.Hv + 7) / 8 * 8;
    const dim3 grid((unsigned)(heads * a.slices)), block(512);
    if constexpr (F32)
        hipLaunchKernelGGL(delta_chunks_f32_kernel<DT>, grid, block, 0, s, a);
    else if (vec)
        hipLaunchKernelGGL((delta_chunks_kernel<DT, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((delta_chunks_kernel<DT, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

bool delta_chunked_supports(int64_t tokens, int num_seqs, int Hk, int Hv, int Dk, int Dv)
{
    // The threads of both grids stay below 2^32.
    return Dk <= 128 && tokens / C + num_seqs < (1 << 24) && ((int64_t)num_seqs * Hv + 8) * ((Dv + 15) / 16) < (1 << 23);
}

template <int DT, bool F32>
static int64_t chunk_bytes(int Hk, int Hv)
{
    return (int64_t)Hk * Space<DT, F32>::KEY + (int64_t)Hv * Space<DT, F32>::VAL;
}

int64_t delta_chunked_workspace(int64_t tokens, int num_seqs, int Hk, int Hv, int Dk, conv_dtype dtype)
{
    const int64_t numbers = tokens / C + num_seqs;
    if (dtype == CONV_F32)
        return numbers * (Dk <= 64 ? chunk_bytes<1, true>(Hk, Hv) : chunk_bytes<2, true>(Hk, Hv));
    return numbers * (Dk <= 64 ? chunk_bytes<1, false>(Hk, Hv) : chunk_bytes<2, false>(Hk, Hv));
}

hipError_t launch_delta_chunked(const DeltaProblem &p, hipStream_t s)
{
    if (p.dtype == CONV_F32)
        return p.Dk <= 64 ? launch<1, true>(p, s) : launch<2, true>(p, s);
    return p.Dk <= 64 ? launch<1, false>(p, s) : launch<2, false>(p, s);
}

}  // namespace convfwd
