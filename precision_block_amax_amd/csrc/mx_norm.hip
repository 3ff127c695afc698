// mx_norm.hip -- layer norm and RMS norm for gfx950, forward (to bf16, or
// straight to the quantized operand of the next product) and backward.
//
// Forward: y = (x - mean) * rstd * weight + bias, one row at a time held whole
// in the registers of T threads (U vectors of 8 elements each), so x is read
// once: its sum, then the sum of the squares of x - mean, then y.  The sums
// are fp32 over fp32 values; taking the squares after the mean loses nothing
// to cancellation.  Vector v of a row is thread v % T's, so that 4 (16)
// neighbouring lanes hold a block of 32 (128) and its amax is a DPP maximum.
//
// Backward, with xh = (x - mean) * rstd, g = dy * weight:
//   dx = rstd * (g - mean(g) - xh * mean(g * xh)),
//   dweight = sum_rows dy * xh, dbias = sum_rows dy.
// dx takes a row per T threads as above.  The sums over rows are taken in two
// steps in a fixed order (chunks of rows into the workspace, then the chunks),
// so that the same inputs give the same bits.
//
// All of it is bound by memory: 2 bytes read and 2 (1 for FP8) written per
// element forward, 4 read and 2 written backward.
#include "mx_block_util.h"

namespace mx {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

// sum over the T threads of a row: T = 64 is one wave; above, the waves meet in `s`
// (one slot per wave, a slot array of its own for each use between two barriers)
template <int T>
__device__ __forceinline__ float row_sum(float v, float *s) {
    v = wave_sum(v);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < T / 64; i++) v += s[i];
    }
    return v;
}

// n (up to 8) parameters at index c, as fp32; `other` where there are none
__device__ __forceinline__ void load_param8(float (&w)[8], const void *p, bool bf16, int c, int n, float other) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = other;
    } else if (bf16) {
        uint32_t t[4];
        load8_bf16(t, reinterpret_cast<const uint16_t *>(p) + c, n);
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = (i & 1) ? bf16_hi(t[i >> 1]) : bf16_lo(t[i >> 1]);
    } else {
        const float *q = reinterpret_cast<const float *>(p) + c;
        if (n >= 8) {
            __builtin_memcpy(w, q, 32);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) w[i] = i < n ? q[i] : 0.f;
        }
    }
}

__device__ __forceinline__ void store8_bf16(uint16_t *p, const float (&y)[8], int n) {
    uint32_t t[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        typedef float v2f __attribute__((ext_vector_type(2)));
        t[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{y[2 * k], y[2 * k + 1]}, v2bf));
    }
    if (n >= 8) {
        __builtin_memcpy(p, t, 16);
    } else {
        for (int i = 0; i < n; i++) p[i] = (uint16_t)(t[i >> 1] >> (16 * (i & 1)));
    }
}

// T threads and 8 T U >= cols elements per row; a workgroup of max(T, 256) threads
template <int T, int U, int TO, int F>
__global__ __launch_bounds__((T < 256 ? 256 : T)) void k_norm(NormArgs a) {
    constexpr int NT = T < 256 ? 256 : T, RPW = NT / T;
    __shared__ float s0[NT / 64], s1[NT / 64];
    const int t = threadIdx.x % T;
    const float rn = 1.0f / (float)a.cols;
    for (int64_t row0 = (int64_t)blockIdx.x * RPW; row0 < a.rows; row0 += (int64_t)gridDim.x * RPW) {
        const int64_t row = row0 + threadIdx.x / T;
        const bool live = row < a.rows;  // with one wave per row the others go on; with more RPW is 1
        float y[U][8];
        const uint16_t *px = a.x + row * a.ldx;
        uint32_t w[U][4];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int n = a.cols - 8 * (u * T + t);
            w[u][0] = w[u][1] = w[u][2] = w[u][3] = 0;
            if (live && n > 0) load8_bf16(w[u], px + 8 * (u * T + t), n);
        }
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int i = 0; i < 8; i++) {
                y[u][i] = (i & 1) ? bf16_hi(w[u][i >> 1]) : bf16_lo(w[u][i >> 1]);
                sum += y[u][i];
            }
        float mean = 0.f;
        if (!a.rms) {
            mean = row_sum<T>(sum, s0) * rn;
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int n = a.cols - 8 * (u * T + t);
#pragma unroll
                for (int i = 0; i < 8; i++) y[u][i] = i < n ? y[u][i] - mean : 0.f;
            }
        }
        float sq = 0.f;
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int i = 0; i < 8; i++) sq = __builtin_fmaf(y[u][i], y[u][i], sq);
        const float var = row_sum<T>(sq, s1) * rn;
        const float rstd = 1.0f / __builtin_sqrtf(var + a.eps);
        if (live && t == 0) {
            if (a.mean && !a.rms) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = 8 * (u * T + t), n = a.cols - c;
            float wt[8], b[8];
            if (n > 0) {
                load_param8(wt, a.weight, a.param_bf16, c, n, 1.f);
                load_param8(b, a.bias, a.param_bf16, c, n, 0.f);
            }
#pragma unroll
            for (int i = 0; i < 8; i++) y[u][i] = i < n ? __builtin_fmaf(y[u][i] * rstd, wt[i], b[i]) : 0.f;
            if constexpr (TO == TO_BF16) {
                if (live && n > 0) store8_bf16(reinterpret_cast<uint16_t *>(a.out) + row * a.ld_out + c, y[u], n);
            } else {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 8; i++) m = umax(m, __float_as_uint(y[u][i]) & 0x7FFFFFFFu);
                m = TO == TO_BLOCK ? row16_max(m) : quad_max(m);
                uint8_t *q = reinterpret_cast<uint8_t *>(a.out) + row * a.ld_out + (F == E2M1 ? c / 2 : c);
                if constexpr (TO == TO_BLOCK) {
                    float sc, inv;
                    bool ok;
                    block_scale<F>(m, sc, inv, ok);
                    const uint32_t lo = block_cvt4<F>(y[u][0], y[u][1], y[u][2], y[u][3], inv, ok);
                    const uint32_t hi = block_cvt4<F>(y[u][4], y[u][5], y[u][6], y[u][7], inv, ok);
                    if (live && n > 0) {
                        store8(q, lo, hi, n);
                        if ((t & 15) == 0)
                            reinterpret_cast<float *>(a.scales)[(int64_t)(c / kBlk) * a.ld_scales + row] = sc;
                    }
                } else {
                    const bool ok = m < 0x7F800000u;
                    const int e = scale_exp_f32<F>(ok ? m : 0u);
                    const float sc = __builtin_amdgcn_ldexpf(1.0f, e);
                    if (live && n > 0) {  // cols is a multiple of 32: whole vectors
                        if constexpr (F == E2M1) {
                            const uint32_t v = ok ? cvt8_fp4(y[u], sc) : 0u;
                            __builtin_memcpy(q, &v, 4);
                        } else {
                            const float lim = __builtin_amdgcn_ldexpf(MaxNormal<F>::v, e);
                            const uint32_t v[2] = {ok ? cvt4_fp8<F>(y[u][0], y[u][1], y[u][2], y[u][3], sc, lim) : 0u,
                                                   ok ? cvt4_fp8<F>(y[u][4], y[u][5], y[u][6], y[u][7], sc, lim) : 0u};
                            __builtin_memcpy(q, v, 8);
                        }
                        if ((t & 3) == 0)
                            reinterpret_cast<uint8_t *>(a.scales)[row * a.ld_scales + c / 32] = (uint8_t)(ok ? e + 127 : 0xFF);
                    }
                }
            }
        }
        // the slots of the sums are written again for the next row
        if (T > 64 && row0 + (int64_t)gridDim.x * RPW < a.rows) __syncthreads();
    }
}

template <int T, int U, int TO, int F>
hipError_t launch_norm_tu(const NormArgs &a, hipStream_t s) {
    constexpr int NT = T < 256 ? 256 : T, RPW = NT / T;
    const int64_t wgs = (a.rows + RPW - 1) / RPW;
    const dim3 grid((unsigned)(wgs < (1 << 20) ? wgs : (1 << 20))), block(NT);
    hipLaunchKernelGGL((k_norm<T, U, TO, F>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <int TO, int F>
hipError_t launch_norm_to(const NormArgs &a, hipStream_t s) {
    if (a.cols <= 512) return launch_norm_tu<64, 1, TO, F>(a, s);
    if (a.cols <= 1024) return launch_norm_tu<64, 2, TO, F>(a, s);
    if (a.cols <= 2048) return launch_norm_tu<256, 1, TO, F>(a, s);
    if (a.cols <= 4096) return launch_norm_tu<256, 2, TO, F>(a, s);
    if (a.cols <= 8192) return launch_norm_tu<256, 4, TO, F>(a, s);
    if (a.cols <= 16384) return launch_norm_tu<1024, 2, TO, F>(a, s);
    return launch_norm_tu<1024, 4, TO, F>(a, s);
}

// ---------------------------------------------------------------------------
template <int T, int U>
__global__ __launch_bounds__((T < 256 ? 256 : T)) void k_norm_dx(NormBwdArgs a) {
    constexpr int NT = T < 256 ? 256 : T, RPW = NT / T;
    __shared__ float s0[NT / 64], s1[NT / 64];
    const int t = threadIdx.x % T;
    const float rn = 1.0f / (float)a.cols;
    for (int64_t row0 = (int64_t)blockIdx.x * RPW; row0 < a.rows; row0 += (int64_t)gridDim.x * RPW) {
        const int64_t row = row0 + threadIdx.x / T;
        const bool live = row < a.rows;
        uint32_t wx[U][4], wd[U][4];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = 8 * (u * T + t), n = a.cols - c;
#pragma unroll
            for (int k = 0; k < 4; k++) wx[u][k] = wd[u][k] = 0;
            if (live && n > 0) {
                load8_bf16(wx[u], a.x + row * a.ldx + c, n);
                load8_bf16(wd[u], a.dy + row * a.lddy + c, n);
            }
        }
        const float rstd = live ? a.rstd[row] : 0.f;
        const float mean = live && !a.rms ? a.mean[row] : 0.f;
        float sg = 0.f, sgx = 0.f;
        float g[U][8], xh[U][8];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = 8 * (u * T + t), n = a.cols - c;
            float wt[8];
            if (n > 0) load_param8(wt, a.weight, a.param_bf16, c, n, 1.f);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float xv = (i & 1) ? bf16_hi(wx[u][i >> 1]) : bf16_lo(wx[u][i >> 1]);
                const float dv = (i & 1) ? bf16_hi(wd[u][i >> 1]) : bf16_lo(wd[u][i >> 1]);
                xh[u][i] = i < n ? (xv - mean) * rstd : 0.f;
                g[u][i] = i < n ? dv * wt[i] : 0.f;
                sg += g[u][i];
                sgx = __builtin_fmaf(g[u][i], xh[u][i], sgx);
            }
        }
        const float mg = a.rms ? 0.f : row_sum<T>(sg, s0) * rn;
        const float mgx = row_sum<T>(sgx, s1) * rn;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = 8 * (u * T + t), n = a.cols - c;
            if (!live || n <= 0) continue;
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; i++) d[i] = (g[u][i] - mg - xh[u][i] * mgx) * rstd;
            store8_bf16(a.dx + row * a.lddx + c, d, n);
        }
        // the slots of the sums are written again for the next row
        if (T > 64 && row0 + (int64_t)gridDim.x * RPW < a.rows) __syncthreads();
    }
}

constexpr int kPartCols = 512;  // columns per workgroup of the partial sums, 8 per lane

// sums of chunk blockIdx.y of the rows: ws[chunk][0 or 1][cols]
__global__ __launch_bounds__(256) void k_norm_dparam(NormBwdArgs a, int64_t rows_per_chunk) {
    __shared__ float s[3][2][kPartCols];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * kPartCols + 8 * lane, n = a.cols - c;
    const int64_t r0 = (int64_t)blockIdx.y * rows_per_chunk, r1 = min(a.rows, r0 + rows_per_chunk);
    float dw[8], db[8];
#pragma unroll
    for (int i = 0; i < 8; i++) dw[i] = db[i] = 0.f;
    if (n > 0) {
        for (int64_t r = r0 + wave; r < r1; r += 4) {
            uint32_t wx[4], wd[4];
            load8_bf16(wx, a.x + r * a.ldx + c, n);
            load8_bf16(wd, a.dy + r * a.lddy + c, n);
            const float rstd = a.rstd[r], mean = a.rms ? 0.f : a.mean[r];
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float xv = (i & 1) ? bf16_hi(wx[i >> 1]) : bf16_lo(wx[i >> 1]);
                const float dv = (i & 1) ? bf16_hi(wd[i >> 1]) : bf16_lo(wd[i >> 1]);
                dw[i] = __builtin_fmaf(dv, (xv - mean) * rstd, dw[i]);
                db[i] += dv;
            }
        }
    }
    if (wave > 0) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            s[wave - 1][0][8 * lane + i] = dw[i];
            s[wave - 1][1][8 * lane + i] = db[i];
        }
    }
    __syncthreads();
    if (wave == 0) {
        float *d = a.ws + (int64_t)blockIdx.y * 2 * a.cols + c;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            if (i >= n) break;
            d[i] = dw[i] + s[0][0][8 * lane + i] + s[1][0][8 * lane + i] + s[2][0][8 * lane + i];
            d[a.cols + i] = db[i] + s[0][1][8 * lane + i] + s[1][1][8 * lane + i] + s[2][1][8 * lane + i];
        }
    }
}

// the chunks' sums: 64 columns of one of the two gradients per workgroup
__global__ __launch_bounds__(256) void k_norm_dparam_sum(NormBwdArgs a, int chunks) {
    __shared__ float s[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float *out = blockIdx.y ? a.db : a.dw;
    if (!out) return;  // uniform
    float v = 0.f;
    if (c < a.cols)
        for (int k = wave; k < chunks; k += 4) v += a.ws[((int64_t)k * 2 + blockIdx.y) * a.cols + c];
    s[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && c < a.cols) out[c] = (s[0][lane] + s[1][lane]) + (s[2][lane] + s[3][lane]);
}

// chunks of rows of the partial sums: 16 rows at least, 128 chunks at most
int64_t dparam_chunks(int64_t rows) {
    const int64_t n = (rows + 15) / 16;
    return n < 128 ? n : 128;
}

template <int T, int U>
hipError_t launch_dx(const NormBwdArgs &a, hipStream_t s) {
    constexpr int NT = T < 256 ? 256 : T, RPW = NT / T;
    const int64_t wgs = (a.rows + RPW - 1) / RPW;
    const dim3 grid((unsigned)(wgs < (1 << 20) ? wgs : (1 << 20))), block(NT);
    hipLaunchKernelGGL((k_norm_dx<T, U>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs &a, int to, int fmt, hipStream_t s) {
    if (to == TO_BF16) return launch_norm_to<TO_BF16, E4M3>(a, s);
    if (to == TO_BLOCK)
        return fmt == E4M3 ? launch_norm_to<TO_BLOCK, E4M3>(a, s) : launch_norm_to<TO_BLOCK, E5M2>(a, s);
    switch (fmt) {
    case E4M3: return launch_norm_to<TO_MX, E4M3>(a, s);
    case E5M2: return launch_norm_to<TO_MX, E5M2>(a, s);
    default: return launch_norm_to<TO_MX, E2M1>(a, s);
    }
}

int64_t norm_backward_workspace(int64_t rows, int64_t cols) { return dparam_chunks(rows) * 2 * cols; }

hipError_t launch_norm_backward(const NormBwdArgs &a, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (a.rows > 0) {
        if (a.cols <= 512) e = launch_dx<64, 1>(a, s);
        else if (a.cols <= 1024) e = launch_dx<64, 2>(a, s);
        else if (a.cols <= 2048) e = launch_dx<256, 1>(a, s);
        else if (a.cols <= 4096) e = launch_dx<256, 2>(a, s);
        else if (a.cols <= 8192) e = launch_dx<256, 4>(a, s);
        else if (a.cols <= 16384) e = launch_dx<1024, 2>(a, s);
        else e = launch_dx<1024, 4>(a, s);
        if (e != hipSuccess) return e;
    }
    if (!a.dw && !a.db) return e;
    const int64_t chunks = dparam_chunks(a.rows);
    if (chunks > 0) {
        const dim3 grid((unsigned)((a.cols + kPartCols - 1) / kPartCols), (unsigned)chunks);
        hipLaunchKernelGGL(k_norm_dparam, grid, dim3(256), 0, s, a, (a.rows + chunks - 1) / chunks);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k_norm_dparam_sum, dim3((unsigned)((a.cols + 63) / 64), 2), dim3(256), 0, s, a, (int)chunks);
    return hipGetLastError();
}

}  // namespace mx
