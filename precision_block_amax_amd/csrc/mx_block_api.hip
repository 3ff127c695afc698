// mx_block_api.hip -- the extern "C" entry points of the block-128 FP8
// operators and of the norm (include/mx.h).  As in mx_api.hip: every argument
// is validated on the host before the first HIP call, then the device is
// checked and the kernels are launched on the caller's stream; nothing is
// allocated and no call synchronizes.
#include <math.h>

#include "mx_block_internal.h"
#include "mx_check.h"

namespace {

using namespace mx;

constexpr int64_t kMaxDim = (int64_t)1 << 31;

bool fp8(int f) { return f == MX_E4M3 || f == MX_E5M2; }
bool type_ok(int t) { return t == MX_OUT_F32 || t == MX_OUT_BF16; }
int64_t blocks(int64_t n) { return (n + kBlk - 1) / kBlk; }

// `rows` rows of `width` used bytes, one every `stride` bytes (0: a single row); `n` bytes from the first of them to the
// end of the last, -1 if that leaves 64 bits
struct Range {
    const void *p;
    int64_t n, width, stride;
};
Range run(const void *p, int64_t n) { return {p, n, n, 0}; }
// row stride ld, `width` used, in units of `size` bytes
Range rows_at(const void *p, int64_t rows, int64_t ld, int64_t width, int64_t size) {
    if (rows <= 0 || width <= 0) return run(p, 0);
    if (width > INT64_MAX / size) return run(p, -1);
    if (rows == 1) return run(p, width * size);
    if (rows - 1 > (INT64_MAX / size - width) / ld) return run(p, -1);
    return {p, ((rows - 1) * ld + width) * size, width * size, ld * size};
}
// no byte belongs to both: their whole extents are disjoint, or the rows of one lie in the gaps of the other's
bool disjoint(const Range &a, const Range &b) {
    if (!overlap(a.p, a.n, b.p, b.n)) return true;
    return a.stride > 0 && a.stride == b.stride && interleaved(a.p, a.width, b.p, b.width, a.stride);
}
// every range exists (n >= 0) and no range from `first_out` on overlaps another one
mx_status_t check_ranges(const Range *r, int count, int first_out) {
    for (int i = 0; i < count; i++)
        if (r[i].n < 0) return MX_ERR_INVALID_ARG;
    for (int i = first_out; i < count; i++)
        for (int j = 0; j < i; j++)
            if (!disjoint(r[i], r[j])) return MX_ERR_INVALID_ARG;
    return MX_OK;
}

// one output form: codes [n x k] with k the reduction dimension, scales [blocks(k)][n or blocks(n)]
mx_status_t check_form(int64_t n, int64_t k, bool tile, int fmt, const void *codes, int64_t ld_codes,
                       const float *scales, int64_t ld_scales, Range *r) {
    if (!fp8(fmt) || ld_codes < k || ld_scales < (tile ? blocks(n) : n)) return MX_ERR_INVALID_ARG;
    if (n == 0 || k == 0) return MX_OK;
    if (!codes || !scales) return MX_ERR_INVALID_ARG;
    r[0] = rows_at(codes, n, ld_codes, k, 1);
    r[1] = rows_at(scales, blocks(k), ld_scales, tile ? blocks(n) : n, 4);
    return MX_OK;
}

mx_status_t block_quantize(const void *x, int64_t rows, int64_t cols, int64_t ldx, bool tile, const BlockForm *row,
                           const BlockForm *tr, void *stream) {
    if (rows < 0 || cols < 0 || ldx < cols) return MX_ERR_INVALID_ARG;
    Range r[5];
    int n = 1;
    mx_status_t st;
    if (row) {
        st = check_form(rows, cols, tile, row->fmt, row->codes, row->ld_codes, row->scales, row->ld_scales, r + n);
        if (st != MX_OK) return st;
        n += 2;
    }
    if (tr) {
        st = check_form(cols, rows, tile, tr->fmt, tr->codes, tr->ld_codes, tr->scales, tr->ld_scales, r + n);
        if (st != MX_OK) return st;
        n += 2;
    }
    if (rows == 0 || cols == 0) return MX_OK;
    if (!x) return MX_ERR_INVALID_ARG;
    r[0] = rows_at(x, rows, ldx, cols, 2);
    if ((st = check_ranges(r, n, 1)) != MX_OK) return st;
    // one workgroup of 256 threads per tile, counted in 32 bits
    if (rows > kMaxDim || cols > kMaxDim || blocks(rows) * blocks(cols) >= ((int64_t)1 << 24)) return MX_ERR_UNSUPPORTED;
    if ((st = check_device()) != MX_OK) return st;
    const BlockForm none{nullptr, 0, nullptr, 0, 0};
    return launched(launch_block_quantize((const uint16_t *)x, rows, cols, ldx, tile, row ? *row : none, tr ? *tr : none,
                                          (hipStream_t)stream));
}

mx_status_t check_norm(const void *x, int64_t rows, int64_t cols, int64_t ldx, int param, int kind) {
    if (rows < 0 || cols < 0 || ldx < cols || !type_ok(param) || (kind != MX_NORM_LAYER && kind != MX_NORM_RMS))
        return MX_ERR_INVALID_ARG;
    if (rows > 0 && cols > 0 && !x) return MX_ERR_INVALID_ARG;
    if (rows > 0 && (cols > kNormMaxCols || rows > kMaxDim)) return MX_ERR_UNSUPPORTED;
    return MX_OK;
}

mx_status_t norm(const void *x, int64_t rows, int64_t cols, int64_t ldx, const void *weight, const void *bias,
                 int param, int kind, float eps, int to, int fmt, void *out, int64_t ld_out, int64_t out_width,
                 int64_t out_size, void *scales, int64_t ld_scales, const Range &scale_range, float *mean, float *rstd,
                 void *stream) {
    mx_status_t st = check_norm(x, rows, cols, ldx, param, kind);
    if (st != MX_OK) return st;
    if (!(eps >= 0.0f) || isinf(eps)) return MX_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return MX_OK;
    if (!out || (to != TO_BF16 && !scales)) return MX_ERR_INVALID_ARG;
    const int64_t ps = param == MX_OUT_BF16 ? 2 : 4;
    if (kind == MX_NORM_RMS) mean = nullptr;
    const Range r[7] = {rows_at(x, rows, ldx, cols, 2),
                        run(weight, weight ? cols * ps : 0),
                        run(bias, bias ? cols * ps : 0),
                        rows_at(out, rows, ld_out, out_width, out_size),
                        scale_range,
                        run(mean, mean ? rows * 4 : 0),
                        run(rstd, rstd ? rows * 4 : 0)};
    if ((st = check_ranges(r, 7, 3)) != MX_OK) return st;
    if ((st = check_device()) != MX_OK) return st;
    const NormArgs a{(const uint16_t *)x, rows,   ldx,    (int)cols, weight, bias,     param == MX_OUT_BF16,
                     kind == MX_NORM_RMS, eps,    mean,   rstd,      out,    ld_out,   scales,
                     ld_scales};
    return launched(launch_norm(a, to, fmt, (hipStream_t)stream));
}

// mx_block_gemm_sums with its enum arguments already read as ints
mx_status_t block_gemm(const void *a_codes, int64_t lda, const float *a_scales, int64_t ldsa, int fa,
                       const void *b_codes, int64_t ldb, const float *b_scales, int64_t ldsb, int fb, int b_tile,
                       int64_t M, int64_t N, int64_t K, void *c, int out, int64_t ldc, int sums, void *stream) {
    if (M < 0 || N < 0 || K < 0 || !fp8(fa) || !fp8(fb) || !type_ok(out) || (b_tile != 0 && b_tile != 1))
        return MX_ERR_INVALID_ARG;
    if (sums != MX_SUMS_F32 && (sums != MX_SUMS_FP8 || out != MX_OUT_BF16)) return MX_ERR_INVALID_ARG;
    const int64_t nb = b_tile ? blocks(N) : N;
    if (lda < K || ldb < K || ldsa < M || ldsb < nb || ldc < N) return MX_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return MX_OK;
    if (!c || (K > 0 && (!a_codes || !a_scales || !b_codes || !b_scales))) return MX_ERR_INVALID_ARG;
    const Range r[5] = {rows_at(a_codes, M, lda, K, 1), rows_at(a_scales, blocks(K), ldsa, M, 4),
                        rows_at(b_codes, N, ldb, K, 1), rows_at(b_scales, blocks(K), ldsb, nb, 4),
                        rows_at(c, M, ldc, N, out == MX_OUT_BF16 ? 2 : 4)};
    mx_status_t st = check_ranges(r, 5, 4);
    if (st != MX_OK) return st;
    // sizes in 31 bits, K rounded up to whole blocks too; at most 2^22 workgroups of up to 512 threads
    if (M >= kMaxDim || N >= kMaxDim || K > kMaxDim - kBlk || blocks(M) * blocks(N) >= ((int64_t)1 << 22))
        return MX_ERR_UNSUPPORTED;
    if ((st = check_device()) != MX_OK) return st;
    BlockGemmArgs g{(const uint8_t *)a_codes, (const uint8_t *)b_codes, a_scales, b_scales, c, lda, ldb, ldsa, ldsb, ldc,
                    (int)M, (int)N, (int)K, out == MX_OUT_BF16, 0, 0};
    return launched(launch_block_gemm(g, fa, fb, b_tile != 0, sums == MX_SUMS_FP8, (hipStream_t)stream));
}

}  // namespace

extern "C" {

mx_status_t mx_block_quantize(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx, mx_format_t fmt,
                              mx_block_mode_t mode, void *codes, int64_t ld_codes, float *scales, int64_t ld_scales,
                              void *stream) {
    const int m = raw(mode);
    if (m < MX_BLOCK_ROW || m > MX_BLOCK_TILE_TRANSPOSE) return MX_ERR_INVALID_ARG;
    const BlockForm f{(uint8_t *)codes, ld_codes, scales, ld_scales, raw(fmt)};
    const bool tr = m == MX_BLOCK_TRANSPOSE || m == MX_BLOCK_TILE_TRANSPOSE;
    return block_quantize(x_bf16, rows, cols, ldx, m >= MX_BLOCK_TILE, tr ? nullptr : &f, tr ? &f : nullptr, stream);
}

mx_status_t mx_block_quantize_dual(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx, int tile,
                                   mx_format_t fmt_row, void *codes_row, int64_t ld_codes_row, float *scales_row,
                                   int64_t ld_scales_row, mx_format_t fmt_t, void *codes_t, int64_t ld_codes_t,
                                   float *scales_t, int64_t ld_scales_t, void *stream) {
    if (tile != 0 && tile != 1) return MX_ERR_INVALID_ARG;
    const BlockForm r{(uint8_t *)codes_row, ld_codes_row, scales_row, ld_scales_row, raw(fmt_row)};
    const BlockForm t{(uint8_t *)codes_t, ld_codes_t, scales_t, ld_scales_t, raw(fmt_t)};
    return block_quantize(x_bf16, rows, cols, ldx, tile != 0, &r, &t, stream);
}

mx_status_t mx_block_gemm(const void *a_codes, int64_t lda, const float *a_scales, int64_t ldsa, mx_format_t fa,
                          const void *b_codes, int64_t ldb, const float *b_scales, int64_t ldsb, mx_format_t fb,
                          int b_tile, int64_t M, int64_t N, int64_t K, void *c, mx_out_t out, int64_t ldc,
                          void *stream) {
    const int o = raw(out);
    return block_gemm(a_codes, lda, a_scales, ldsa, raw(fa), b_codes, ldb, b_scales, ldsb, raw(fb), b_tile, M, N, K, c,
                      o, ldc, o == MX_OUT_BF16 ? MX_SUMS_FP8 : MX_SUMS_F32, stream);
}

mx_status_t mx_block_gemm_sums(const void *a_codes, int64_t lda, const float *a_scales, int64_t ldsa, mx_format_t fa,
                               const void *b_codes, int64_t ldb, const float *b_scales, int64_t ldsb, mx_format_t fb,
                               int b_tile, int64_t M, int64_t N, int64_t K, void *c, mx_out_t out, int64_t ldc,
                               mx_sums_t sums, void *stream) {
    return block_gemm(a_codes, lda, a_scales, ldsa, raw(fa), b_codes, ldb, b_scales, ldsb, raw(fb), b_tile, M, N, K, c,
                      raw(out), ldc, raw(sums), stream);
}

mx_status_t mx_layer_norm(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx, const void *weight,
                          const void *bias, mx_out_t param, mx_norm_t kind, float eps, void *y_bf16, int64_t ldy,
                          float *mean, float *rstd, void *stream) {
    if (ldy < cols) return MX_ERR_INVALID_ARG;
    return norm(x_bf16, rows, cols, ldx, weight, bias, raw(param), raw(kind), eps, TO_BF16, 0, y_bf16, ldy, cols, 2,
                nullptr, 0, run(nullptr, 0), mean, rstd, stream);
}

mx_status_t mx_layer_norm_quantize(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx, const void *weight,
                                   const void *bias, mx_out_t param, mx_norm_t kind, float eps, mx_format_t fmt,
                                   void *codes, void *scales, float *mean, float *rstd, void *stream) {
    const int f = raw(fmt);
    if (!fmt_ok(f) || cols < 0 || cols % 32 != 0 || rows < 0) return MX_ERR_INVALID_ARG;
    const int64_t cb = code_bytes(cols, f), sb = cols / 32;
    return norm(x_bf16, rows, cols, ldx, weight, bias, raw(param), raw(kind), eps, TO_MX, f, codes, cb, cb, 1, scales,
                sb, rows_at(scales, rows, sb, sb, 1), mean, rstd, stream);
}

mx_status_t mx_layer_norm_block_quantize(const void *x_bf16, int64_t rows, int64_t cols, int64_t ldx,
                                         const void *weight, const void *bias, mx_out_t param, mx_norm_t kind,
                                         float eps, mx_format_t fmt, void *codes, int64_t ld_codes, float *scales,
                                         int64_t ld_scales, float *mean, float *rstd, void *stream) {
    const int f = raw(fmt);
    if (!fp8(f) || cols < 0 || rows < 0 || ld_codes < cols || ld_scales < rows) return MX_ERR_INVALID_ARG;
    return norm(x_bf16, rows, cols, ldx, weight, bias, raw(param), raw(kind), eps, TO_BLOCK, f, codes, ld_codes, cols,
                1, scales, ld_scales, rows_at(scales, blocks(cols), ld_scales, rows, 4), mean, rstd, stream);
}

int64_t mx_layer_norm_backward_workspace(int64_t rows, int64_t cols) {
    return rows <= 0 || cols <= 0 ? 0 : norm_backward_workspace(rows, cols) * 4;
}

mx_status_t mx_layer_norm_backward(const void *dy_bf16, int64_t lddy, const void *x_bf16, int64_t ldx, int64_t rows,
                                   int64_t cols, const void *weight, mx_out_t param, mx_norm_t kind,
                                   const float *mean, const float *rstd, void *dx_bf16, int64_t lddx, float *dweight,
                                   float *dbias, void *workspace, int64_t workspace_bytes, void *stream) {
    const int p = raw(param), k = raw(kind);
    mx_status_t st = check_norm(x_bf16, rows, cols, ldx, p, k);
    if (st != MX_OK) return st;
    if (lddy < cols || lddx < cols) return MX_ERR_INVALID_ARG;
    if (cols == 0 || (rows == 0 && !dweight && !dbias)) return MX_OK;
    if (cols > kMaxDim) return MX_ERR_UNSUPPORTED;  // (no rows)
    if (rows > 0 && (!dy_bf16 || !rstd || !dx_bf16 || (k == MX_NORM_LAYER && !mean))) return MX_ERR_INVALID_ARG;
    const int64_t need = dweight || dbias ? mx_layer_norm_backward_workspace(rows, cols) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need || (uintptr_t)workspace % 16 != 0)) return MX_ERR_INVALID_ARG;
    const Range r[9] = {rows_at(dy_bf16, rows, lddy, cols, 2),
                        rows_at(x_bf16, rows, ldx, cols, 2),
                        run(weight, weight ? cols * (p == MX_OUT_BF16 ? 2 : 4) : 0),
                        run(mean, k == MX_NORM_LAYER ? rows * 4 : 0),
                        run(rstd, rows * 4),
                        rows_at(dx_bf16, rows, lddx, cols, 2),
                        run(dweight, dweight ? cols * 4 : 0),
                        run(dbias, dbias ? cols * 4 : 0),
                        run(workspace, need)};
    if ((st = check_ranges(r, 9, 5)) != MX_OK) return st;
    if ((st = check_device()) != MX_OK) return st;
    const NormBwdArgs a{(const uint16_t *)dy_bf16, (const uint16_t *)x_bf16, rows, lddy, ldx, lddx, (int)cols, weight,
                        p == MX_OUT_BF16, k == MX_NORM_RMS, mean, rstd, (uint16_t *)dx_bf16, dweight, dbias,
                        (float *)workspace};
    return launched(launch_norm_backward(a, (hipStream_t)stream));
}

}  // extern "C"
