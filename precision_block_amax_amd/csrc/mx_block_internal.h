// mx_block_internal.h -- launchers of the block-128 FP8 operators and of the
// norm, shared by their translation units.  Not part of the public ABI.
#pragma once
#include "mx_internal.h"

namespace mx {

constexpr int kBlk = 128;                     // block (and tile) edge
constexpr float kAmaxFloor = 0x1p-100f;       // smallest amax a scale is made from
// Largest value of the element format
template <int F> constexpr float block_fmax() { return F == E4M3 ? 448.0f : 57344.0f; }

// One output form of a block-128 quantization; codes == nullptr: not written
struct BlockForm {
    uint8_t *codes;
    int64_t ld_codes;
    float *scales;
    int64_t ld_scales;
    int fmt;
};

// row: the form with cols as the reduction dimension, tr: the transposed one.
// At least one of them is wanted; rows, cols > 0.
hipError_t launch_block_quantize(const uint16_t *x, int64_t rows, int64_t cols, int64_t ldx, bool tile,
                                 const BlockForm &row, const BlockForm &tr, hipStream_t stream);

struct BlockGemmArgs {
    const uint8_t *a, *b;
    const float *as, *bs;
    void *c;
    int64_t lda, ldb, ldsa, ldsb, ldc;
    int M, N, K;
    bool c_bf16;
    int tiles_m, tiles_n;
};

// M, N > 0; K == 0 clears C.  fp8_sums: blocks' sums by the FP8 instruction (C in bf16 only), else in fp32
hipError_t launch_block_gemm(const BlockGemmArgs &g, int fa, int fb, bool b_tile, bool fp8_sums, hipStream_t stream);

struct NormArgs {
    const uint16_t *x;
    int64_t rows, ldx;
    int cols;
    const void *weight, *bias;  // may be nullptr
    bool param_bf16, rms;
    float eps;
    float *mean, *rstd;         // may be nullptr
    // outputs: y (bf16), or codes and scales
    void *out;
    int64_t ld_out;
    void *scales;
    int64_t ld_scales;
};

constexpr int kNormMaxCols = 32768;  // a row is held in the registers of one workgroup
enum NormTo : int { TO_BF16 = 0, TO_BLOCK = 1, TO_MX = 2 };

hipError_t launch_norm(const NormArgs &a, int to, int fmt, hipStream_t stream);

struct NormBwdArgs {
    const uint16_t *dy, *x;
    int64_t rows, lddy, ldx, lddx;
    int cols;
    const void *weight;
    bool param_bf16, rms;
    const float *mean, *rstd;
    uint16_t *dx;
    float *dw, *db;             // may be nullptr
    float *ws;
};

// floats of workspace launch_norm_backward uses where a gradient of a parameter is wanted
int64_t norm_backward_workspace(int64_t rows, int64_t cols);
hipError_t launch_norm_backward(const NormBwdArgs &a, hipStream_t stream);

}  // namespace mx
