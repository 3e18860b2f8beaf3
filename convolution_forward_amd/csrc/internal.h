// Internal declarations shared by the host dispatcher and the kernel files.
// Nothing here is part of the public ABI (include/convfwd.h is).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "convfwd.h"

namespace convfwd {

// A validated dense problem: NHWC X with element strides, KKIO F, NHWC Y.
struct DenseProblem {
    const void *X;
    int64_t xs[4];
    const void *F;
    const float *bias;
    void *Y;
    int64_t ys[4];
    int N, H, W, Cin, KH, KW, Cout, Ho, Wo;
    conv_dtype xdt, ydt;
    // Window: stride, padding before each axis (the padding after only
    // shapes Ho and Wo), dilation, groups. The lecture's operator is
    // sh = sw = dh = dw = groups = 1, pt = pl = 0.
    int sh, sw, pt, pl, dh, dw, groups;
};

// True for the lecture's restricted operator (unit stride, no padding, no
// dilation, one group).
inline bool plain_window(const DenseProblem &p)
{
    return p.sh == 1 && p.sw == 1 && p.pt == 0 && p.pl == 0 && p.dh == 1 && p.dw == 1 && p.groups == 1 &&
           p.Ho == p.H - p.KH + 1 && p.Wo == p.W - p.KW + 1;
}

// A validated depthwise problem: contiguous NCHW X, [C*mult,KH,KW] w, NCHW Y.
struct DwProblem {
    const float *X;
    const float *w;
    const float *bias;
    float *Y;
    int N, C, H, W, mult, KH, KW, sh, sw, ph, pw, dh, dw, Ho, Wo;
    int pb, pr;         // padding after each axis (ph, pw are the padding before)
    conv_dw_mode mode;
};

// Dense kernels.
hipError_t launch_dense_direct(const DenseProblem &p, hipStream_t s);
bool dense_band_supports(const DenseProblem &p);
bool dense_pw_supports(const DenseProblem &p);
hipError_t launch_dense_pw(const DenseProblem &p, hipStream_t s);
hipError_t launch_dense_band(const DenseProblem &p, int gpack, hipStream_t s);
bool dense_mfma_bf16_supports(const DenseProblem &p);
hipError_t launch_dense_mfma_bf16(const DenseProblem &p, hipStream_t s);
bool dense_gemm_bf16_supports(const DenseProblem &p);
hipError_t launch_dense_gemm_bf16(const DenseProblem &p, hipStream_t s);
bool dense_mfma_f32_supports(const DenseProblem &p);
hipError_t launch_dense_mfma_f32(const DenseProblem &p, hipStream_t s);
bool dense_gemm_f32_supports(const DenseProblem &p);
bool dense_f32x6_supports(const DenseProblem &p);
hipError_t launch_dense_f32x6(const DenseProblem &p, hipStream_t s);
hipError_t launch_dense_gemm_f32(const DenseProblem &p, hipStream_t s);

// Depthwise kernels.
hipError_t launch_dw_direct(const DwProblem &p, hipStream_t s);
bool dw_tiled_supports(const DwProblem &p);
bool dw_pad_supports(const DwProblem &p);
bool dw_waves_supports(const DwProblem &p);
hipError_t launch_dw_waves(const DwProblem &p, hipStream_t s);
bool dw_planes_supports(const DwProblem &p);
bool dw_rows_supports(const DwProblem &p);
hipError_t launch_dw_rows(const DwProblem &p, hipStream_t s);
hipError_t launch_dw_planes(const DwProblem &p, hipStream_t s);
hipError_t launch_dw_pad(const DwProblem &p, hipStream_t s);
hipError_t launch_dw_tiled(const DwProblem &p, hipStream_t s);

// A validated explicit patch-matrix problem: NHWC X with element strides,
// cols contiguous [N*Ho*Wo, KH*KW*Cin] of the same dtype.
struct Im2colProblem {
    const void *X;
    int64_t xs[4];
    void *cols;
    int N, H, W, Cin, KH, KW, Ho, Wo;
    int sh, sw, pt, pl, dh, dw;
    conv_dtype dtype;
};

hipError_t launch_im2col(const Im2colProblem &p, hipStream_t s);

// ---- Token-mixer operators (mixer_api.cpp validates, one file each) --------

// A validated RMS norm with 8-bit output.
struct NormProblem {
    const void *x, *residual, *weight;
    void *h, *q;
    float *scale;
    int64_t xs, rs, hs, qs;     // row strides in elements
    int64_t rows;
    int width;
    float eps;
    conv_dtype dtype, qdt;
};

hipError_t launch_rms_norm_q8(const NormProblem &p, hipStream_t s);

// A validated product of 8-bit operands.
struct MatmulQ8Problem {
    const void *x, *w;
    const float *xscale, *wscale, *bias;
    void *y;
    int64_t xs, ws, ys;         // row strides in elements
    int64_t M;
    int N, K;
    conv_dtype qdt, ydt;
};

hipError_t launch_matmul_q8_direct(const MatmulQ8Problem &p, hipStream_t s);
bool matmul_q8_tiled_supports(const MatmulQ8Problem &p);
hipError_t launch_matmul_q8(const MatmulQ8Problem &p, hipStream_t s);

// Packed sequences and their state slots (device arrays; seq_offsets NULL =
// equal lengths, slots NULL = slot n for sequence n).
struct Sequences {
    const int32_t *offsets;
    const int32_t *slots;
    int num_slots;
    int num_seqs;
    int64_t tokens;
    int64_t each;               // tokens / num_seqs, the length of each where offsets is NULL
};

// A validated causal convolution over packed sequences.
struct Causal1dProblem {
    const void *x, *w;
    const float *bias;
    void *y;
    int64_t xs, ys;             // row strides in elements
    const void *state_in;
    void *state_out;
    Sequences seq;
    int channels, taps, silu;
    conv_dtype dtype;
};

bool causal1d_supports(const Causal1dProblem &p);
hipError_t launch_causal1d(const Causal1dProblem &p, hipStream_t s);

// A validated gated delta rule.
struct DeltaProblem {
    const void *q, *k, *v;
    const float *g, *beta;
    void *o;
    int64_t qst, qsh, kst, ksh, vst, vsh, ost, osh;     // token and head strides in elements
    const float *state_in;
    float *state_out;
    Sequences seq;
    void *workspace;
    int Hk, Hv, Dk, Dv;
    float scale;
    int normalize;
    conv_dtype dtype;
};

bool delta_direct_supports(int64_t tokens, int num_seqs, int Hv, int Dk, int Dv);
hipError_t launch_delta_direct(const DeltaProblem &p, hipStream_t s);
bool delta_chunked_supports(int64_t tokens, int num_seqs, int Hk, int Hv, int Dk, int Dv);
int64_t delta_chunked_workspace(int64_t tokens, int num_seqs, int Hk, int Hv, int Dk, conv_dtype dtype);
hipError_t launch_delta_chunked(const DeltaProblem &p, hipStream_t s);

// Validated head norms and rotation. Hk == 0: no keys.
struct RotaryProblem {
    const void *q, *k;
    void *q_out, *k_out;
    int64_t qst, qsh, kst, ksh, qot, qoh, kot, koh;     // token and head strides in elements
    const void *qweight, *kweight;                      // NULL: no norm
    const void *positions;                              // int64 if wide, else int32
    const float *frequencies;
    int64_t tokens;
    int wide, Hq, Hk, D, rotated, interleaved;
    float eps, scale;
    conv_dtype dtype;
};

bool rotary_supports(int64_t tokens, int heads, int D);
hipError_t launch_rotary(const RotaryProblem &p, hipStream_t s);

// A validated selective scan with a decay for each channel and state.
struct ScanProblem {
    const void *x, *dt, *b, *c, *gate;
    const float *a, *skip, *bias;
    void *y;
    int64_t xs, dts, gs, ys;                            // row strides in elements
    int64_t bst, bsg, cst, csg;                         // token and group strides in elements
    const float *state_in;
    float *state_out;
    Sequences seq;
    void *workspace;
    int channels, groups, N, softplus;
    conv_dtype dtype;
};

bool scan_direct_supports(int num_seqs, int channels, int N);
hipError_t launch_scan_direct(const ScanProblem &p, hipStream_t s);
bool scan_tiled_supports(int64_t tokens, int num_seqs, int channels, int groups, int N);
int64_t scan_tiled_workspace(int64_t tokens, int num_seqs, int channels, int groups, int N);
hipError_t launch_scan_tiled(const ScanProblem &p, hipStream_t s);

// A validated selective scan with one decay a head.
struct HeadScanProblem {
    const void *x, *dt, *b, *c, *gate;
    const float *a, *skip, *bias;
    void *y;
    int64_t xst, xsh, gst, gsh, yst, ysh;               // token and head strides in elements
    int64_t dts;                                        // token stride of dt
    int64_t bst, bsg, cst, csg;                         // token and group strides in elements
    const float *state_in;
    float *state_out;
    Sequences seq;
    void *workspace;
    int H, P, groups, N, softplus;
    conv_dtype dtype;
};

bool heads_direct_supports(int num_seqs, int H, int P, int N);
hipError_t launch_heads_direct(const HeadScanProblem &p, hipStream_t s);
bool heads_chunked_supports(int64_t tokens, int num_seqs, int H, int P, int groups, int N, conv_dtype dtype);
int64_t heads_chunked_workspace(int64_t tokens, int num_seqs, int H, int P, int groups, int N, conv_dtype dtype);
hipError_t launch_heads_chunked(const HeadScanProblem &p, hipStream_t s);

// Streaming copies used for bandwidth / counter calibration.
hipError_t launch_copy_bytes(const void *src, void *dst, int64_t bytes, hipStream_t s);
hipError_t launch_copy_wide(const void *src, void *dst, int64_t bytes, hipStream_t s);

}  // namespace convfwd
