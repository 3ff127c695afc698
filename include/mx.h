/*
 * mx.h -- C ABI of libmx: OCP-MX micro-scaling quantization, the fixed-sign
 * 32-point block-Hadamard rotation, and the MX-scaled GEMM, for AMD gfx950
 * (Instinct MI355X).
 *
 * What the calls compute, and where it is stated:
 *   - MX micro-scaling (FP4-training article on hzrcw.cc, section 02: the tensor
 *     is cut into small blocks, each with its own dynamic scaling exponent;
 *     MXFP4 is an OCP open format, section 04).  Block size 32 along the
 *     reduction dimension (MindSpeed-LLM FSDP2 quantization page: recipe
 *     dynamic_MX-1-1-32 and --model.quant_block_size 32).
 *   - Element formats E4M3 and E5M2 (Lumen page, section 1: E4M3 for
 *     precision, E5M2 for range) and E2M1 (MXFP4), OCP encodings: E4M3 "FN"
 *     (bias 7, max 448, no infinities), E5M2 (bias 15, max normal 57344),
 *     E2M1 (bias 1, max 6).  Shared scale: one E8M0 byte per block,
 *       S = clamp(floor(log2 amax) - emax, -127, 127) + 127,
 *     emax = 8 (E4M3), 15 (E5M2), 2 (E2M1); elements are v * 2^-(S-127),
 *     rounded to nearest (ties to even) and saturated to +-max normal.
 *   - The deterministic fixed-sign Hadamard rotation on the weight-gradient
 *     path (FP4-training article, section 02: one fixed orthogonal transform
 *     in place of random rotations), applied along tokens before the FP4
 *     quantization of both weight-gradient operands.
 *   - Products by expert (MindSpeed-LLM FSDP2 page: quantization of the experts'
 *     layers, quantize.moe.mx, and Qwen3-30B-A3B, whose attention normalises the
 *     heads of queries and keys) and rotary positions with Llama-3.1's frequency
 *     bands: the block-128 calls by group and the calls on heads below.
 *   - The quantized GEMMs of a linear layer (FP4-training article, section
 *     02: forward, activation-gradient and weight-gradient GEMMs), which the
 *     Primus page names as the dominant training cost (GEMM tuning section).
 *
 * Conventions shared by every call:
 *   - All data pointers are DEVICE pointers, allocated and freed by the
 *     caller.  The library allocates nothing and keeps no per-call state.
 *   - `stream` is a hipStream_t passed as void*; NULL is the default (null)
 *     stream.  Calls are asynchronous on that stream and never synchronize.
 *   - Inputs are read only.  Outputs are overwritten completely (no
 *     accumulation).  Inputs and outputs must not overlap.
 *   - bf16 inputs are row-major with a leading dimension `ldx` (elements
 *     between the starts of consecutive rows, ldx >= cols).
 *     (The calls by group leave what belongs to no group as it was.)
 *   - Outputs are dense row-major (the _panels calls and pair modes write
 *     their codes in the K-panel layout described before them instead):
 *       FP8 codes   : one byte per element;
 *       E2M1 codes  : two elements per byte, element 2i in bits 3:0 and
 *                     element 2i+1 in bits 7:4;
 *       scales      : one E8M0 byte per 32-element block.
 *   - A block that holds an Inf or NaN gets scale 0xFF (E8M0 NaN) and all
 *     element codes 0.  An all-zero block gets scale 0x00.  The sign of zero
 *     is kept (-0 -> 0x80 for FP8, 0x8 for E2M1).
 *   - A size of 0 is a valid empty call: nothing is read or written (except
 *     mx_gemm and the block-128 products with K == 0, which write C = 0, and the
 *     norms' backward passes without rows, which write zero gradients of the
 *     parameters), and pointers may be NULL.
 *
 * Errors (no call throws, no call aborts):
 *   MX_ERR_INVALID_ARG  bad argument, detected on the host before any HIP
 *                       call: NULL pointer with a non-empty size, negative
 *                       size, a blocked dimension not a multiple of 32,
 *                       ldx < cols, ldc < N, unknown enum value, or
 *                       operand and output buffers that overlap.
 *   MX_ERR_UNSUPPORTED  the current device is not gfx950, or an index range
 *                       exceeds what the kernels address (more than 2^31
 *                       blocks or rows in one call).
 *   MX_ERR_HIP          a HIP runtime call or kernel launch failed.
 *   Faults inside a kernel surface at the caller's next synchronization.
 */
#ifndef MX_H
#define MX_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MX_OK = 0,
    MX_ERR_INVALID_ARG = 1,
    MX_ERR_UNSUPPORTED = 2,
    MX_ERR_HIP = 3
} mx_status_t;

typedef enum {
    MX_E4M3 = 0, /* FP8 1-4-3, bias 7, max 448       */
    MX_E5M2 = 1, /* FP8 1-5-2, bias 15, max 57344    */
    MX_E2M1 = 2  /* FP4 1-2-1, bias 1, max 6, packed */
} mx_format_t;

typedef enum {
    MX_OUT_F32 = 0, /* fp32 output                          */
    MX_OUT_BF16 = 1 /* bf16 output, fp32 result rounded RNE */
} mx_out_t;

/*
 * mx_quantize -- row mode.  Block b of row r is x[r, 32b .. 32b+31].
 *   x_bf16  [rows x ldx] bf16, reads the first `cols` of each row
 *   cols    multiple of 32
 *   codes   [rows x cols] bytes (E4M3/E5M2) or [rows x cols/2] (E2M1)
 *   scales  [rows x cols/32] E8M0 bytes
 * This is the Fprop operand quantizer (activations and weights stored with
 * the reduction dimension contiguous) and the Dgrad quantizer of the output
 * gradient.
 * Defined by: FP4-training article on hzrcw.cc, section 02 (MX blocks, each
 * with its own dynamic power-of-two exponent, on the forward and
 * activation-gradient GEMM operands); MindSpeed-LLM FSDP2 page, section
 * "三步启用 MXFP8 低精度训练" (block size 32 along the reduction dimension);
 * Lumen page, section 1 (the E4M3 and E5M2 element formats).
 */
mx_status_t mx_quantize(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx,
                        mx_format_t fmt, void *codes, void *scales, void *stream);

/*
 * mx_quantize_transpose -- transposed mode.  Block b of column c is
 * x[32b .. 32b+31, c]; it becomes block b of output row c, so the output is
 * the MX form of x^T with `rows` as its contiguous (reduction) dimension.
 *   rows    multiple of 32
 *   codes   [cols x rows] bytes (E4M3/E5M2) or [cols x rows/2] (E2M1)
 *   scales  [cols x rows/32]
 * Used for operands whose reduction dimension is strided in storage: the
 * weight in Dgrad (reduction over N_out) and, without rotation, the two
 * weight-gradient operands (reduction over tokens).
 * Defined by: FP4-training article on hzrcw.cc, section 02 (the
 * activation-gradient and weight-gradient GEMMs quantize their operands
 * along the GEMM's own reduction dimension), with the block and formats of
 * mx_quantize.
 */
mx_status_t mx_quantize_transpose(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx,
                                  mx_format_t fmt, void *codes, void *scales, void *stream);

/*
 * mx_hadamard32_quantize -- transposed mode after the fixed-sign block
 * rotation.  For each column c and each 32-row block b, with
 * x_i = x[32b + i, c] widened to fp32:
 *     x_i <- -x_i  where bit i of sign_mask is set,
 *     five butterfly stages h = 1, 2, 4, 8, 16, each replacing
 *     (x_j, x_{j+h}) by (x_j + x_{j+h}, x_j - x_{j+h}) for every j with
 *     (j & h) == 0, one fp32 rounding per operation,
 *     y_i = x_i * c with c = 0x3E3504F3 = RN_fp32(1/sqrt(32)),
 * i.e. y = c * H32 * diag(s) * x with H32 the Sylvester-Hadamard matrix.
 * y (fp32, no bf16 rounding) is then quantized as block b of output row c,
 * with the same output layout as mx_quantize_transpose.  Rotation blocks
 * coincide with the MX blocks.  sign_mask = 0 is the plain Sylvester
 * rotation.  Results are bit-identical for every launch configuration.
 * Defined by: FP4-training article on hzrcw.cc, section 02 (one fixed,
 * deterministic Hadamard rotation of both weight-gradient operands along
 * tokens before the FP4 quantization, in place of random rotations).  The
 * sign vector, stage order, constant and fp32 arithmetic are the readings
 * written out above; the page gives the transform only in words.
 */
mx_status_t mx_hadamard32_quantize(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx,
                                   uint32_t sign_mask, mx_format_t fmt, void *codes, void *scales,
                                   void *stream);

/*
 * mx_quantize_transpose_sr -- mx_quantize_transpose (rotate = 0) or
 * mx_hadamard32_quantize (rotate = 1, with sign_mask) with stochastic instead
 * of nearest rounding of the elements; same scales, same layout.  Stochastic
 * rounding is the randomised cast that the FP4-training article on hzrcw.cc
 * (section 01) names as the common remedy for FP4 training, against which it
 * argues for the deterministic rotation; it is here for that comparison.
 * Each element q = y * 2^-e (y the block value after the optional rotation,
 * e the block's scale exponent) lies between grid neighbours lo <= |q| < hi
 * and rounds up iff its 32-bit random word r < floor(2^32 (|q|-lo)/(hi-lo)),
 * so the up-probability is the fractional position to 32 bits; magnitudes
 * at or above the largest normal saturate; signs are kept.  Random words:
 * element t of output row c is element i = c * rows + t of the Philox4x32-10
 * stream (Salmon, Moraes, Dror, Shaw, SC 2011): word i mod 4 of the block at
 * counter (i / 4 low word, i / 4 high word, 0, 0) and key (seed low word,
 * seed high word).  The result depends only on x and seed, not on the launch
 * configuration.
 *   rotate  0 or 1
 * Sizes, layout, ownership and errors as mx_quantize_transpose.
 */
mx_status_t mx_quantize_transpose_sr(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx, int rotate,
                                     uint32_t sign_mask, uint64_t seed, mx_format_t fmt, void *codes, void *scales,
                                     void *stream);

/*
 * mx_quantize_dual -- the row form and the transposed form of x from one
 * read of x: codes_row / scales_row exactly as mx_quantize(x, fmt_row), and
 * codes_t / scales_t exactly as mx_quantize_transpose(x, fmt_t) (rotate = 0)
 * or mx_hadamard32_quantize(x, sign_mask, fmt_t) (rotate = 1).
 *   rows, cols  both multiples of 32
 *   rotate      0 or 1
 * A linear layer needs both forms of its activations, output gradients and
 * weights: the row form for Fprop and Dgrad, the transposed (for the
 * gradients, rotated) form for Dgrad's weight and for the weight gradient
 * (FP4-training article on hzrcw.cc, section 02).  The four output buffers
 * must not overlap each other or x.
 */
mx_status_t mx_quantize_dual(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx,
                             mx_format_t fmt_row, void *codes_row, void *scales_row,
                             mx_format_t fmt_t, int rotate, uint32_t sign_mask, void *codes_t,
                             void *scales_t, void *stream);

typedef enum {
    MX_PAIR_ROW = 0,              /* as mx_quantize                               */
    MX_PAIR_TRANSPOSE = 1,        /* as mx_quantize_transpose                     */
    MX_PAIR_HADAMARD = 2,         /* as mx_hadamard32_quantize (sign_mask)        */
    MX_PAIR_TRANSPOSE_PANELS = 3, /* as mx_quantize_transpose_panels              */
    MX_PAIR_HADAMARD_PANELS = 4   /* as mx_hadamard32_quantize_panels (sign_mask) */
} mx_pair_mode_t;

/*
 * mx_quantize_pair -- the two operands of one GEMM in one launch.  x0 (rows0
 * x cols0, leading dimension ldx0) goes to codes0 / scales0 and x1 to codes1
 * / scales1, each exactly as the single call of `mode` would quantize it:
 * same format `fmt`, the same sign_mask for the rotated modes (ignored
 * otherwise), and per tensor the sizes, layouts, rules and errors of that
 * call.  The GEMMs of a linear layer take both operands in the same form
 * (FP4-training article on hzrcw.cc, section 02: Fprop X and W in row mode,
 * Wgrad dY and X rotated along tokens).  One launch for both saves one
 * launch's start-up and drain.  On MI355X that is 4-6% of the time for
 * the Llama-3.1-8B operand pairs.  Where the two need different
 * kernel variants (a strided or unaligned tensor), the call runs the two
 * single quantizations one after the other on `stream`; an empty tensor is
 * skipped.  Neither tensor's outputs may overlap the other tensor's input
 * or outputs (the two inputs may overlap: they are only read).
 */
mx_status_t mx_quantize_pair(mx_pair_mode_t mode, mx_format_t fmt, uint32_t sign_mask,
                             const void *x0, int64_t rows0, int64_t cols0, int64_t ldx0, void *codes0,
                             void *scales0, const void *x1, int64_t rows1, int64_t cols1, int64_t ldx1,
                             void *codes1, void *scales1, void *stream);

/*
 * mx_gemm -- C[m, n] = sum_k A[m, k] * B[n, k] over two MX operands, both
 * with the reduction dimension K contiguous ("TN"):
 *   a_codes [M x K] (FP8) or [M x K/2] (E2M1), a_scales [M x K/32]
 *   b_codes [N x K] (FP8) or [N x K/2] (E2M1), b_scales [N x K/32]
 *   A[m, k] = decode(code) * 2^(S - 127), same for B
 *   K       multiple of 32
 *   c       [M x ldc] fp32 or bf16 (per `out`), ldc >= N
 * E2M1 x E2M1 products are formed by the gfx950 block-scaled matrix
 * instruction (64 elements of K per step, exact), pairs with an FP8 operand
 * by the bf16 matrix instruction on codes converted exactly to bf16 against
 * a per-row reference scale; partial sums are accumulated in fp32, so
 * |C - sum| <= 1e-5 * sum |A[m, k] * B[n, k]|.  Fprop: A = X, B = W.
 * Dgrad: A = dY, B = W^T (from mx_quantize_transpose).  Wgrad: A = dY^T,
 * B = X^T (both from mx_hadamard32_quantize or mx_quantize_transpose).
 * Any pair of formats is accepted.
 * Defined by: FP4-training article on hzrcw.cc, section 02 (the forward,
 * activation-gradient and weight-gradient GEMMs on MX operands); Primus page,
 * sections "性能瓶颈分析" and "GEMM 调优" (GEMM as the dominant training cost).
 * A scale byte 0xFF (E8M0 NaN) makes every output element it contributes to
 * NaN.
 */
mx_status_t mx_gemm(const void *a_codes, const void *a_scales, mx_format_t fa,
                    const void *b_codes, const void *b_scales, mx_format_t fb,
                    int64_t M, int64_t N, int64_t K, void *c, mx_out_t out, int64_t ldc,
                    void *stream);

/*
 * mx_quantize_strided -- mx_quantize with row strides on the outputs: row r's
 * codes go to codes + r * ld_codes and its scales to scales + r * ld_scales
 * (bytes), with ld_codes >= the code bytes of a row (cols, or cols / 2 for
 * E2M1) and ld_scales >= cols / 32.  Codes and scales may share one buffer as
 * long as no byte is written twice: either their extents are disjoint, or
 * ld_codes == ld_scales and each row's scales lie in the gap after its codes.
 *
 * FSDP2 low-precision all-gather payload (MindSpeed-LLM FSDP2 page, section
 * "第 3 步：开启低精度 All-Gather", weights sharded along dim 0 as its
 * "注意事项" requires): a rank quantizes its slab of weight rows [rows x K]
 * (x = its rows, ldx = the full row) into ONE buffer of rows
 *     [ codes (code_bytes(K)) | scales (K / 32) | 0 .. 15 bytes unused ],
 * i.e. codes = payload, scales = payload + code_bytes(K), ld_codes =
 * ld_scales = code_bytes(K) + K / 32 rounded up to a multiple of 16 (no
 * padding when K % 512 == 0; 1.03125 bytes per element for FP8, 0.53125 for
 * E2M1, against 2 for bf16).  K blocks never cross rows, so the
 * ranks' payloads concatenated in rank order -- what an all-gather of one
 * buffer per rank delivers -- are exactly the same layout for the whole
 * weight, bit-identical to quantizing it in one call, and mx_gemm_strided
 * takes them as an operand with those two strides, without a copy.
 * Errors as mx_quantize.
 */
mx_status_t mx_quantize_strided(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx, mx_format_t fmt,
                                void *codes, int64_t ld_codes, void *scales, int64_t ld_scales, void *stream);

/*
 * mx_gemm_strided -- mx_gemm on operands whose rows are strided: row m of A's
 * codes starts at a_codes + m * lda and its scales at a_scales + m * ldsa
 * (bytes), likewise for B with ldb and ldsb; lda >= code bytes of K
 * elements and a multiple of 16 (code rows are read with 16-byte loads; the
 * dense stride always is one), ldsa >= K / 32 (any value).  mx_gemm is the
 * case lda = code bytes of K and ldsa = K / 32.  Used for the gathered FSDP2 payload (see
 * mx_quantize_strided) and for operands that are row slices of larger
 * buffers.  Scale strides that are multiples of 16 bytes, with 16-byte
 * aligned code and dword-aligned scale pointers, keep the pipelined kernel
 * (K % 512 == 0); other strides run the general kernels.
 * Same tolerance as mx_gemm; with the same kernel the results are
 * bit-identical to mx_gemm's on the same values.
 */
mx_status_t mx_gemm_strided(const void *a_codes, int64_t lda, const void *a_scales, int64_t ldsa, mx_format_t fa,
                            const void *b_codes, int64_t ldb, const void *b_scales, int64_t ldsb, mx_format_t fb,
                            int64_t M, int64_t N, int64_t K, void *c, mx_out_t out, int64_t ldc, void *stream);

/*
 * K-panel layout of MX codes -- an alternative storage order of the same
 * codes, chosen by the library for its own transposed quantizers and GEMM
 * (no page prescribes a layout).  The codes of R rows of K elements are K / P
 * panels of R rows x 128 bytes, P = 256 elements for E2M1 and 128 for
 * E4M3 / E5M2: code byte j (j < 128) of row r in panel p is at
 * codes + p * (R * 128) + r * 128 + j, i.e. bytes [128 p, 128 p + 128) of the
 * dense row r.  Same total size as the dense layout; scales stay dense
 * ([R x K/32]).  A transposed quantizer writes each workgroup's codes as
 * whole 32 KiB runs in this order (256 runs of 128 bytes in the dense one),
 * and the GEMM reads both layouts at about the same speed.
 */
typedef enum {
    MX_LAYOUT_ROWS = 0,   /* dense row-major codes, as every other call */
    MX_LAYOUT_PANELS = 1  /* K-panel layout above                        */
} mx_layout_t;

/*
 * mx_quantize_transpose_panels, mx_hadamard32_quantize_panels -- as
 * mx_quantize_transpose and mx_hadamard32_quantize (same codes and scales,
 * same errors), with the codes in the K-panel layout (R = cols output rows,
 * K = rows).  rows must also be a multiple of the panel width: 256 for E2M1,
 * 128 for E4M3 / E5M2 (else MX_ERR_INVALID_ARG).  For callers: the
 * weight-gradient operands that mx_gemm_layout then reads in place.
 */
mx_status_t mx_quantize_transpose_panels(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx,
                                         mx_format_t fmt, void *codes, void *scales, void *stream);
mx_status_t mx_hadamard32_quantize_panels(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx,
                                          uint32_t sign_mask, mx_format_t fmt, void *codes, void *scales,
                                          void *stream);

/*
 * mx_quantize_dual_panels -- mx_quantize_dual (same arguments, codes and
 * scales, same errors) with both forms' codes in the K-panel layout: the
 * row form's (R = rows, K = cols) and the transposed form's (R = cols,
 * K = rows).  cols must be a whole number of fmt_row panels and rows a whole
 * number of fmt_t panels (else MX_ERR_INVALID_ARG).  A workgroup then writes
 * each form as contiguous runs (4 KiB per wave of the row form, 32 KiB of
 * the transposed one).  For callers: a linear layer whose GEMMs all read
 * their operands in place through mx_gemm_layout.
 */
mx_status_t mx_quantize_dual_panels(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx, mx_format_t fmt_row,
                                    void *codes_row, void *scales_row, mx_format_t fmt_t, int rotate,
                                    uint32_t sign_mask, void *codes_t, void *scales_t, void *stream);

/*
 * mx_gemm_layout -- mx_gemm with each operand's codes in the layout given
 * (a_layout, b_layout); scales dense.  With both MX_LAYOUT_ROWS it is
 * mx_gemm.  A K-panel operand needs the pipelined kernel: K a multiple of
 * 512, 16-byte aligned code and dword-aligned scale pointers, the operand's
 * code bytes below 2^31, and, for an E2M1 operand, an E2M1 partner (beside
 * an FP8 operand an E2M1 stage row is 64 bytes, half a panel row); otherwise
 * MX_ERR_UNSUPPORTED.  Any M and N.  Same computation as mx_gemm: on the
 * same values the results are bit-identical to mx_gemm's with dense
 * operands.  Errors otherwise as mx_gemm (MX_ERR_INVALID_ARG for an unknown
 * layout).
 */
mx_status_t mx_gemm_layout(const void *a_codes, mx_layout_t a_layout, const void *a_scales, mx_format_t fa,
                           const void *b_codes, mx_layout_t b_layout, const void *b_scales, mx_format_t fb,
                           int64_t M, int64_t N, int64_t K, void *c, mx_out_t out, int64_t ldc, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Block-128 FP8: one fp32 scale for each block of 128.
 *
 * The other widespread FP8 recipe for a linear layer, beside MX: activations
 * and gradients in blocks of 128 elements along the reduction dimension,
 * weights in 128 x 128 tiles, every block with its own fp32 scale.  Element
 * formats E4M3 and E5M2 (MX_E2M1 is MX_ERR_INVALID_ARG in these calls).
 *   amax  = max(largest |v| of the block, 2^-100)
 *   scale = amax / FMAX                (FMAX = 448 for E4M3, 57344 for E5M2)
 *   code  = cast(clamp(v * (FMAX / amax), -FMAX, FMAX))
 * each operation rounded once in fp32, the cast to nearest, ties to even.  A
 * block that holds an Inf or NaN gets scale NaN and codes 0 (so every product
 * it enters is NaN); an all-zero block gets scale 2^-100 / FMAX and codes +-0.
 * No size has to be a multiple of anything: the last block (tile) of a row
 * may be shorter.
 *
 * Operands.  Codes are rows of bytes, the reduction dimension contiguous, row
 * r at codes + r * ld_codes (any ld_codes >= the row's length; a multiple of
 * 16 with 16-byte aligned codes is the fast case of mx_block_gemm).  Scales
 * have the reduction dimension's blocks outermost: block b of row r (tile b of
 * tile row r) is scales[b * ld_scales + r], ld_scales in floats, >= the number
 * of rows (tile rows).  Bytes between the end of a row and the next row, and
 * floats between the last row's scale and the next block's, are neither read
 * as values nor written.
 *
 * Overlap, in these calls and the norm's below: no byte of an output may be
 * one of another buffer of the call.  Whole extents that are disjoint always
 * qualify; so do two buffers with one row stride in bytes whose rows lie in
 * each other's gaps (a norm's x and y as the halves of wider rows, say).
 */
typedef enum {
    MX_BLOCK_ROW = 0,            /* blocks of 128 along cols; codes [rows x cols]; scales [ceil(cols/128)][rows]  */
    MX_BLOCK_TRANSPOSE = 1,      /* blocks of 128 along rows; codes [cols x rows]; scales [ceil(rows/128)][cols]  */
    MX_BLOCK_TILE = 2,           /* 128 x 128; codes [rows x cols]; scales [ceil(cols/128)][ceil(rows/128)]       */
    MX_BLOCK_TILE_TRANSPOSE = 3  /* 128 x 128; codes [cols x rows]; scales [ceil(rows/128)][ceil(cols/128)]       */
} mx_block_mode_t;

/*
 * mx_block_quantize -- x (bf16, rows x cols, leading dimension ldx) as one
 * block-128 operand, per `mode`.  MX_BLOCK_ROW: activations and output
 * gradients as the left operand of Fprop and Dgrad.  MX_BLOCK_TRANSPOSE: both
 * operands of Wgrad (reduction over tokens).  MX_BLOCK_TILE and its transposed
 * form: the weight in Fprop and Dgrad; the tiles of one weight are the same in
 * both forms, so their codes agree and their scales are each other's
 * transpose.  Codes and scales must not overlap x or each other.
 */
mx_status_t mx_block_quantize(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx, mx_format_t fmt,
                              mx_block_mode_t mode, void *codes, int64_t ld_codes, float *scales, int64_t ld_scales,
                              void *stream);

/*
 * mx_block_quantize_dual -- both forms of x from one read: with tile = 0 the
 * row form (as MX_BLOCK_ROW, format fmt_row) and the transposed form (as
 * MX_BLOCK_TRANSPOSE, fmt_t); with tile = 1 MX_BLOCK_TILE and
 * MX_BLOCK_TILE_TRANSPOSE.  Each exactly as the single call gives it.
 */
mx_status_t mx_block_quantize_dual(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx, int tile,
                                   mx_format_t fmt_row, void *codes_row, int64_t ld_codes_row, float *scales_row,
                                   int64_t ld_scales_row, mx_format_t fmt_t, void *codes_t, int64_t ld_codes_t,
                                   float *scales_t, int64_t ld_scales_t, void *stream);

/*
 * mx_block_gemm -- C[m, n] = sum over blocks b of
 *     sa[b][m] * sb[b][n] * sum_{k in block b} A[m, k] * B[n, k]
 * with A [M x K] in blocks of 128 along K and B [N x K] likewise (b_tile = 0)
 * or in 128 x 128 tiles (b_tile = 1: sb[b][n / 128]).  Any M, N and K (K = 0
 * writes C = 0; M or N of 2^31 and more, K above 2^31 - 128 and 2^22 or more
 * tiles of 128 x 128 are MX_ERR_UNSUPPORTED); lda, ldb in bytes, ldsa, ldsb in
 * floats, c [M x ldc] per `out`, ldc >= N.  Every block's sum is multiplied by
 * its scales and added to an fp32 accumulator.
 *   MX_OUT_F32   every product is exact and sums are fp32: |C - sum| <=
 *                (130 + ceil(K / 128)) * 2^-24 * sum |terms|, which is one
 *                rounding for each of a block's additions, for its scales and
 *                for each block's addition to the rest (1e-5 up to K = 4736;
 *                random data stays within it far beyond).  The codes travel as
 *                fp16 (exact) through the fp16 matrix instruction.
 *   MX_OUT_BF16  the FP8 matrix instruction, at twice that rate.  It adds the
 *                32 products of a step in a window that ends 2^-13 below the
 *                largest, so a block's sum may be off by 2^-8 of its sum of
 *                |terms| in the worst case (2^-11 and less on random data):
 *                below the result's own rounding to bf16 unless the sum cancels
 *                far.  Where that matters, MX_OUT_F32 or mx_block_gemm_sums.
 * Products of two scales outside fp32's range are Inf or 0, those below 2^-126
 * keep the bits that a subnormal number has.  A NaN scale makes
 * every element of C that it contributes to NaN; NaN and Inf codes behave as
 * these values.  Fast are operands whose rows are aligned to 16 bytes (any K;
 * as the quantizers' callers lay them out); others take a general kernel, at
 * about two thirds of the speed.  A row's last 16 aligned bytes are read whole,
 * its bytes past K not used.
 */
mx_status_t mx_block_gemm(const void *a_codes, int64_t lda, const float *a_scales, int64_t ldsa, mx_format_t fa,
                          const void *b_codes, int64_t ldb, const float *b_scales, int64_t ldsb, mx_format_t fb,
                          int b_tile, int64_t M, int64_t N, int64_t K, void *c, mx_out_t out, int64_t ldc,
                          void *stream);

/*
 * mx_block_gemm_sums -- mx_block_gemm with the choice of how a block's sum is
 * formed: MX_SUMS_F32 in fp32, as MX_OUT_F32 has it, for either output (bf16 is
 * that result rounded once); MX_SUMS_FP8 by the FP8 matrix instruction, as
 * MX_OUT_BF16 has it (with MX_OUT_F32 it is MX_ERR_INVALID_ARG).
 */
typedef enum {
    MX_SUMS_FP8 = 0, /* a window of 13 bits within 32 products, fp32 from block to block */
    MX_SUMS_F32 = 1  /* exact products, fp32 sums; half the matrix rate                  */
} mx_sums_t;
mx_status_t mx_block_gemm_sums(const void *a_codes, int64_t lda, const float *a_scales, int64_t ldsa, mx_format_t fa,
                               const void *b_codes, int64_t ldb, const float *b_scales, int64_t ldsb, mx_format_t fb,
                               int b_tile, int64_t M, int64_t N, int64_t K, void *c, mx_out_t out, int64_t ldc,
                               mx_sums_t sums, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Block-128 products by group: a layer of experts, each with a weight of its own.
 *
 * Rows (tokens, sorted by expert) are in `groups` groups, given by the ends of
 * their ranges in DEVICE memory, so that nothing waits for the host to learn them:
 * group i is the rows from ends[i - 1] (0 for the first) to ends[i] - 1, ends not
 * decreasing and at most `rows`.  Groups may be empty; rows from the last end on
 * belong to none, and what is at their place in an output is left as it was.  (An
 * end below the one before it or above `rows` is taken as these, but see
 * mx_block_gemm_grouped_k; nothing outside the buffers is touched whatever ends
 * holds.)  At most 2^16 groups.
 *
 * Operands whose reduction dimension is the rows (both of a weight gradient) have
 * their blocks of 128 start anew at every group: block b of the transposed form is
 * 128 rows of one group or its last ones, and the columns behind these hold zeros.
 * mx_block_grouped_cols(rows, groups) columns (a multiple of 128) are enough
 * whatever the groups; blocks behind the last group's are not written.  (0 for
 * sizes that the calls refuse.)
 */
int64_t mx_block_grouped_cols(int64_t rows, int64_t groups);

/*
 * mx_block_quantize_grouped -- the transposed form: codes [cols x ld_codes],
 * ld_codes >= mx_block_grouped_cols(rows, groups); scales [that / 128][ld_scales],
 * ld_scales >= cols.  mx_block_quantize_grouped_dual writes the row form (as
 * MX_BLOCK_ROW) from the same read.  Each block as mx_block_quantize gives it.
 */
mx_status_t mx_block_quantize_grouped(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx, const int32_t *ends,
                                      int64_t groups, mx_format_t fmt, void *codes, int64_t ld_codes, float *scales,
                                      int64_t ld_scales, void *stream);
mx_status_t mx_block_quantize_grouped_dual(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx,
                                           const int32_t *ends, int64_t groups, mx_format_t fmt_row, void *codes_row,
                                           int64_t ld_codes_row, float *scales_row, int64_t ld_scales_row,
                                           mx_format_t fmt_t, void *codes_t, int64_t ld_codes_t, float *scales_t,
                                           int64_t ld_scales_t, void *stream);

/*
 * mx_block_gemm_grouped -- for every row m of group g
 *     C[m, n] = sum over blocks b of sa[b][m] * sb[g][b][n] * sum_{k in b} A[m, k] * B[g][n, k]
 * A [rows x K] and C [rows x N] as in mx_block_gemm_sums; B[g] [N x K] with codes at
 * b_codes + g * ldb_group and scales at b_scales + g * ldsb_group, each as there
 * (b_tile: in 128 x 128 tiles).  The weights of all groups quantized as one matrix
 * of groups * N rows, N a multiple of 128, qualify in both forms: with
 * MX_BLOCK_TILE ldb_group = N * ldb, ldsb_group = N / 128 (ldsb = groups * that);
 * its transposed form is B for the gradient of A: ldb_group = N, ldsb_group = N /
 * 128 * ldsb.  Types, sums, accuracy, limits (for the most tiles that the groups
 * may take) and alignment as in mx_block_gemm_sums; ldb_group a multiple of 16 is
 * the fast case.  K = 0 writes zeros to the groups' rows.
 */
mx_status_t mx_block_gemm_grouped(const void *a_codes, int64_t lda, const float *a_scales, int64_t ldsa, mx_format_t fa,
                                  const void *b_codes, int64_t ldb_group, int64_t ldb, const float *b_scales,
                                  int64_t ldsb_group, int64_t ldsb, mx_format_t fb, int b_tile, const int32_t *ends,
                                  int64_t groups, int64_t rows, int64_t N, int64_t K, void *c, mx_out_t out,
                                  int64_t ldc, mx_sums_t sums, void *stream);

/*
 * mx_block_gemm_grouped_k -- for every group g, its rows being the reduction dimension
 *     C[g][m, n] = sum over the blocks b of g of sa[b][m] * sb[b][n] * sum_{k in b} A[m, k] * B[n, k]
 * A [M x cols] and B [N x cols] as mx_block_quantize_grouped writes them for the same
 * ends, cols a multiple of 128 that holds all the groups' blocks; scales [cols / 128][M]
 * and [.. N].  C[g] [M x ldc] at c + g * ldc_group elements, ldc_group >= (M - 1) *
 * ldc + N.  An empty group's C is zeros.  Types, sums, accuracy and limits (for the
 * tiles of all groups) as in mx_block_gemm_sums, K being the group's rows.
 * This call does not know how many rows the operands were made of: no end may lie
 * above them (it would claim blocks that nobody wrote; what is read stays within cols).
 * mx_block_gemm_grouped_k_rows takes their number, and ends above it as the quantizers do.
 */
mx_status_t mx_block_gemm_grouped_k(const void *a_codes, int64_t lda, const float *a_scales, int64_t ldsa,
                                    mx_format_t fa, const void *b_codes, int64_t ldb, const float *b_scales,
                                    int64_t ldsb, mx_format_t fb, const int32_t *ends, int64_t groups, int64_t M,
                                    int64_t N, int64_t cols, void *c, mx_out_t out, int64_t ldc_group, int64_t ldc,
                                    mx_sums_t sums, void *stream);
mx_status_t mx_block_gemm_grouped_k_rows(const void *a_codes, int64_t lda, const float *a_scales, int64_t ldsa,
                                         mx_format_t fa, const void *b_codes, int64_t ldb, const float *b_scales,
                                         int64_t ldsb, mx_format_t fb, const int32_t *ends, int64_t groups,
                                         int64_t rows, int64_t M, int64_t N, int64_t cols, void *c, mx_out_t out,
                                         int64_t ldc_group, int64_t ldc, mx_sums_t sums, void *stream);

/*
 * ---------------------------------------------------------------------------
 * The norm in front of a linear layer, forward and backward.
 *
 *   mean = sum_j x_j / cols (0 for MX_NORM_RMS),
 *   rstd = 1 / sqrt(sum_j (x_j - mean)^2 / cols + eps),
 *   y_j = (x_j - mean) * rstd * weight_j + bias_j
 * for every row of x (bf16, rows x cols, leading dimension ldx), all in fp32,
 * mean before the squares are summed.  weight and bias: `cols` values of
 * `param` type each, either may be NULL (1 and 0).  mean and rstd: fp32, one
 * per row, for the backward pass; mean is not written for MX_NORM_RMS, either
 * may be NULL.  eps >= 0, finite.  Rows are held whole by a workgroup: cols
 * above 32768 are MX_ERR_UNSUPPORTED.  Sums and squares are fp32 numbers, so
 * values whose squares leave its range (about 1e19 / sqrt(cols)) are not
 * normalised; a constant row with eps = 0 gives NaN.
 */
typedef enum {
    MX_NORM_LAYER = 0, /* mean and variance                        */
    MX_NORM_RMS = 1    /* mean taken as 0: y = x / rms(x) * weight */
} mx_norm_t;

/* y: bf16 [rows x ldy], rounded once, ldy >= cols. */
mx_status_t mx_layer_norm(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx, const void *weight,
                          const void *bias, mx_out_t param, mx_norm_t kind, float eps, void *y_bf16, int64_t ldy,
                          float *mean, float *rstd, void *stream);

/*
 * mx_layer_norm_quantize, mx_layer_norm_block_quantize -- the norm written as
 * the next product's operand, without the trip through bf16: y stays in fp32
 * (no bf16 rounding, as the rotated quantizer's y does) and is quantized as
 * mx_quantize would (any format, cols a multiple of 32, dense codes and
 * scales), or as mx_block_quantize with MX_BLOCK_ROW would (E4M3 or E5M2).
 * Same rules for blocks that hold an Inf or NaN.
 */
mx_status_t mx_layer_norm_quantize(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx, const void *weight,
                                   const void *bias, mx_out_t param, mx_norm_t kind, float eps, mx_format_t fmt,
                                   void *codes, void *scales, float *mean, float *rstd, void *stream);
mx_status_t mx_layer_norm_block_quantize(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx,
                                         const void *weight, const void *bias, mx_out_t param, mx_norm_t kind,
                                         float eps, mx_format_t fmt, void *codes, int64_t ld_codes, float *scales,
                                         int64_t ld_scales, float *mean, float *rstd, void *stream);

/*
 * mx_layer_norm_backward -- with xh = (x - mean) * rstd and g = dy * weight:
 *     dx = rstd * (g - mean_j(g) - xh * mean_j(g * xh))   (RMS: without mean_j(g))
 *     dweight_j = sum over rows of dy * xh,  dbias_j = sum over rows of dy
 * dy, x: bf16; dx: bf16 [rows x lddx], rounded once; dweight, dbias: fp32
 * [cols], overwritten, either may be NULL (rows = 0 writes zeros).  mean (not
 * read for MX_NORM_RMS, may be NULL there) and rstd as the forward call wrote
 * them.  The sums over rows go through `workspace`, workspace_bytes >=
 * mx_layer_norm_backward_workspace(rows, cols) bytes of device memory, 16-byte
 * aligned, that no other call may use until this one has run on the stream;
 * its contents need not be initialised.  It may be NULL if neither gradient is
 * asked for.  Sums are in a fixed order: the same inputs give the same bits.
 */
int64_t mx_layer_norm_backward_workspace(int64_t rows, int64_t cols);
mx_status_t mx_layer_norm_backward(const void *dy_bf16, int64_t lddy, const void *x_bf16, int64_t ldx, int64_t rows,
                                   int64_t cols, const void *weight, mx_out_t param, mx_norm_t kind,
                                   const float *mean, const float *rstd, void *dx_bf16, int64_t lddx, float *dweight,
                                   float *dbias, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Queries and keys after the QKV product: rotary positions, alone or behind an
 * RMS norm of each head, and the backward pass.
 *
 * Queries and keys are two sets of heads of `dim` bf16 elements over the same
 * tokens: element i of head h of token t is at t * ld + h * ld_head + i.  Any
 * strides with tokens outermost (views of one QKV output row included) or heads
 * outermost, no element twice; either set may have no heads.  dim is at most 512,
 * heads at most 2^16 each, tokens at most 2^31 (else MX_ERR_UNSUPPORTED).
 *
 * Rotation.  The first `rot` elements of a head (even, 0 .. dim) form rot / 2
 * pairs, the others stay.  With p the token's position (int32 or int64, negative
 * ones too) and pair i's angle p * freqs[i] (radians, double, device memory):
 *     (a, b) -> (a c - b s, b c + a s),   c, s = scale * (cos, sin)(angle)
 * Angles are taken in fp64 and reduced to one turn there, so far positions lose
 * nothing: |error| <= 2^-21 + |p| freqs[i] 2^-51 radians; the rest is fp32,
 * rounded once to bf16.  inverse = 1 turns by -angle: with the same scale that is
 * the transpose, the backward pass of the rotation.
 */
typedef enum {
    MX_ROPE_HALF = 0,       /* pair i: elements i and i + rot / 2  */
    MX_ROPE_INTERLEAVED = 1 /* pair i: elements 2 i and 2 i + 1    */
} mx_rope_layout_t;
typedef enum {
    MX_POS_I32 = 0,
    MX_POS_I64 = 1
} mx_pos_t;

/*
 * mx_rope_frequencies -- freqs[0 .. rot / 2 - 1] in HOST memory:
 *     theta^(-2 i / rot),
 * for contexts `factor` times as long as the model's first one divided by factor
 * (MX_ROPE_LINEAR), or (MX_ROPE_BANDS) divided only where a pair makes fewer than
 * `low` turns within `original` positions, kept where it makes more than `high`,
 * in between f * keep + f / factor * (1 - keep), keep = (turns - low) / (high -
 * low).  Recipes that also sharpen the attention pass their factor as `scale`.
 * A host function: no GPU is needed.
 */
typedef enum {
    MX_ROPE_PLAIN = 0,  /* factor, low, high and original are not read */
    MX_ROPE_LINEAR = 1, /* low, high and original are not read         */
    MX_ROPE_BANDS = 2
} mx_rope_scaling_t;
mx_status_t mx_rope_frequencies(int64_t rot, double theta, mx_rope_scaling_t scaling, double factor, double low,
                                double high, double original, double *freqs);

mx_status_t mx_rope(const void *q_bf16, int64_t ldq, int64_t ldq_head, int64_t q_heads, const void *k_bf16, int64_t ldk,
                    int64_t ldk_head, int64_t k_heads, int64_t tokens, int64_t dim, const void *positions,
                    mx_pos_t pos_type, const double *freqs, int64_t rot, mx_rope_layout_t layout, float scale,
                    int inverse, void *q_out, int64_t ldqo, int64_t ldqo_head, void *k_out, int64_t ldko,
                    int64_t ldko_head, void *stream);

/*
 * mx_qk_norm_rope -- for every head
 *     xh = x * rstd, rstd = 1 / sqrt(mean(x^2) + eps), y = rotation of xh * weight,
 * weight the `dim` values (of `param` type, NULL: 1) that all query heads, or all
 * key heads, share.  One pass, fp32 until y's one rounding.  eps >= 0, finite;
 * rot = 0 leaves the norm alone (positions and freqs may then be NULL).  Heads of
 * any finite elements are normalised, also where their squares leave fp32's range
 * (which mx_layer_norm's rows may not); a head of zeros with eps = 0 gives NaN.
 */
mx_status_t mx_qk_norm_rope(const void *q_bf16, int64_t ldq, int64_t ldq_head, int64_t q_heads, const void *k_bf16,
                            int64_t ldk, int64_t ldk_head, int64_t k_heads, int64_t tokens, int64_t dim,
                            const void *q_weight, const void *k_weight, mx_out_t param, float eps,
                            const void *positions, mx_pos_t pos_type, const double *freqs, int64_t rot,
                            mx_rope_layout_t layout, float scale, void *q_out, int64_t ldqo, int64_t ldqo_head,
                            void *k_out, int64_t ldko, int64_t ldko_head, void *stream);

/*
 * mx_qk_norm_rope_backward -- with dy the gradient of y, u the transposed rotation
 * of dy and g = u * weight:
 *     dx = rstd * (g - xh * mean(g * xh)),  dweight = sum over tokens and heads of u * xh
 * from x as the forward call read it (rstd is made again; the products g * x are fp32
 * numbers).  dx: bf16, rounded once; dq_weight, dk_weight: fp32 [dim], overwritten
 * (zeros where there are no tokens or no heads), either may be NULL.  workspace as in
 * mx_layer_norm_backward,
 * mx_qk_norm_rope_backward_workspace(tokens, q_heads, k_heads, dim) bytes.  Sums are
 * in a fixed order: the same inputs give the same bits.
 */
int64_t mx_qk_norm_rope_backward_workspace(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim);
mx_status_t mx_qk_norm_rope_backward(const void *dq_bf16, int64_t lddq, int64_t lddq_head, const void *dk_bf16,
                                     int64_t lddk, int64_t lddk_head, const void *q_bf16, int64_t ldq,
                                     int64_t ldq_head, int64_t q_heads, const void *k_bf16, int64_t ldk,
                                     int64_t ldk_head, int64_t k_heads, int64_t tokens, int64_t dim,
                                     const void *q_weight, const void *k_weight, mx_out_t param, float eps,
                                     const void *positions, mx_pos_t pos_type, const double *freqs, int64_t rot,
                                     mx_rope_layout_t layout, float scale, void *dxq_bf16, int64_t lddxq,
                                     int64_t lddxq_head, void *dxk_bf16, int64_t lddxk, int64_t lddxk_head,
                                     float *dq_weight, float *dk_weight, void *workspace, int64_t workspace_bytes,
                                     void *stream);

/* Static, NUL-terminated name of a status code. */
const char *mx_status_string(mx_status_t s);

/* Library version as MAJOR * 10000 + MINOR * 100 + PATCH. */
int mx_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MX_H */
