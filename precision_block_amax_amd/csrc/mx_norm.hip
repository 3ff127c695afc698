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
// One pass: a workgroup takes a chunk of rows, R at a time, each in the
// registers of T threads, and keeps the parameters' sums of its chunk in
// registers too (8 U columns per thread); the chunks' sums go through the
// workspace to a second kernel.  All sums are in a fixed order, so the same
// inputs give the same bits.
//
// Bound by memory: 2 bytes read and 2 (1 for FP8) written per element forward,
// 4 read and 2 written backward; to FP8 the vector units, busy half of the time,
// and the two barriers per row come next.
// Measured with outputs over the same memory call after call: 8192 x 4096 to bf16
// (134 MB) 25.7 us, 5.2 TB/s, to FP8 (102 MB) 23.4 us, 4.4 TB/s; backward (201 MB)
// 47.8 us, 43 of them the first kernel's (outputs in turn, so that nothing stays in
// the last-level cache: 29.6, 27.6, 51.3; to MX E4M3 25.0, E2M1 (85 MB) 19.5);
// without the parameters' sums 42.7.  1001 x 8192 backward (49 MB) 18.8 us: 2 rows
// at a time in a workgroup leave two or three latencies in a row, and the chunks'
// sums are a third of the bytes again.  2048 x 32768 to FP8 (203 MB) 73 us: four
// vectors per thread leave no registers for the next row; backward (403 MB) 189:
// the parameters' kernel reads x and dy a second time.  One row of 4096: 4 us,
// launch and latency.
#include <type_traits>

#include "mx_block_util.h"

namespace mx {
namespace {

// bf16 input larger than half of the 256 MB last-level cache is read past it: less of it would be found there
// than it pushes out.  Through the cache and past it, with outputs over the same memory call after call: 32768 x 4096
// to bf16 115 and 89 us, backward 169 and 140, 8192 x 4096 (67 MB, partly still cached) to bf16 25.7 and 28.2; with
// outputs in turn 114 and 118, 169 and 160, 29.9 and 28.4.
bool past_cache(int64_t rows, int64_t cols) { return rows * cols > (int64_t)1 << 26; }

// sum over the wave, in every lane: within rows of 16 lanes by DPP (neighbours, pairs, mirrored halves,
// mirrored row), then row against row and half against half (one swap gives each side both values)
__device__ __forceinline__ float wave_sum(float v) {
    const auto add = [&](auto ctrl) { v += __uint_as_float(dpp<decltype(ctrl)::value>(__float_as_uint(v))); };
    add(std::integral_constant<int, kDppXor1>{});
    add(std::integral_constant<int, kDppXor2>{});
    add(std::integral_constant<int, kDppHalfMirror>{});
    add(std::integral_constant<int, kDppMirror>{});
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// sum / n, correctly rounded unless it is subnormal: an approximation and one correction by its exact remainder, as
// block_scale (n: a whole number, rn its rounded reciprocal).  sum * rn alone gives constant rows of 896, 1000 or
// 7168 columns a mean beside their value, and y then shows the difference times a very large rstd.  An infinite
// quotient has no remainder.
__device__ __forceinline__ float row_mean(float sum, float n, float rn) {
    const float q = sum * rn;
    const float m = __builtin_fmaf(__builtin_fmaf(-q, n, sum), rn, q);
    return __builtin_fabsf(q) < INFINITY ? m : q;
}

// Parameters of vectors c0 + 8 T u (u < U) as fp32: `other` where there are none, 0 past cols.  Without WHOLE a
// vector that the row's end cuts is taken element by element.  All loads go out before the first is used.
template <bool WHOLE, int T, int U>
__device__ __forceinline__ void load_params(float (&w)[U][8], const void *p, bool bf16, int c0, int cols, float other) {
    if (p && bf16) {
        uint32_t t[U][4];
#pragma unroll
        for (int u = 0; u < U; u++) load_vec<WHOLE>(t[u], reinterpret_cast<const uint16_t *>(p), c0 + 8 * T * u, cols, true);
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int i = 0; i < 8; i++) w[u][i] = (i & 1) ? bf16_hi(t[u][i >> 1]) : bf16_lo(t[u][i >> 1]);
        return;
    }
    if (p) {
        const float *q = reinterpret_cast<const float *>(p);
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = c0 + 8 * T * u;
            if (WHOLE || c + 8 <= cols) {
                __builtin_memcpy(w[u], q + min(c, cols - 8), 32);
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) w[u][i] = q[min(c + i, cols - 1)];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
        for (int i = 0; i < 8; i++) w[u][i] = c0 + 8 * T * u + (WHOLE ? 0 : i) < cols ? (p ? w[u][i] : other) : 0.f;
}

// y as bf16 to columns c .. c + 7 of the row at p, those before cols; WHOLE as in load_vec
template <bool WHOLE>
__device__ __forceinline__ void store_vec(uint16_t *p, const float (&y)[8], int c, int cols) {
    typedef float v2f __attribute__((ext_vector_type(2)));
    uint32_t t[4];
#pragma unroll
    for (int k = 0; k < 4; k++) t[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{y[2 * k], y[2 * k + 1]}, v2bf));
    if (WHOLE ? c < cols : c + 8 <= cols) {
        __builtin_memcpy(reinterpret_cast<uint8_t *>(p) + 2u * (uint32_t)c, t, 16);
    } else if (!WHOLE) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (c + i < cols) p[c + i] = (uint16_t)(t[i >> 1] >> (16 * (i & 1)));
    }
}

// T threads and 8 T U >= cols elements per row, NT / T rows at a time; a workgroup takes the `per` rows from
// blockIdx.x * per on, the next rows' loads under way while it works on these.  T: 4096 columns to FP8, 8192
// rows, took 27 us with 256 threads a row, 28 with 512, 35 with 128 and 39 with a wave (no barriers, but the
// parameters are then read again for every row).  Block scales lie
// rows-innermost, so those of one row are 4-byte stores to as many lines: they are collected in LDS and
// written as runs of the workgroup's rows (8192 x 4096: row by row 34 us, where the bf16 output with a
// third more bytes took 27).
constexpr int kNormRows = 16;  // most rows per workgroup
template <int T, int U, int TO, int F, bool WHOLE, bool PAST>
__global__ __launch_bounds__((T < 256 ? 256 : T)) void k_norm(NormArgs a, int per) {
    constexpr int NT = T < 256 ? 256 : T, RPW = NT / T, W = T / 64;
    // the parameters and the next row fit in registers beside a row (with four vectors per thread they would be
    // spilled: 2048 x 32768 to FP8 97 us with the next row, 68 without)
    constexpr bool KEEP = U <= 2;
    __shared__ float s0[RPW][W], s1[RPW][W];
    __shared__ float sSc[TO == TO_BLOCK ? T * U / 16 * kNormRows : 1];  // [block][row]
    const int t = threadIdx.x % T, grp = __builtin_amdgcn_readfirstlane(threadIdx.x / T);
    const float rn = 1.0f / (float)a.cols;
    const int64_t r0 = (int64_t)blockIdx.x * per;
    const int count = (int)min((int64_t)per, a.rows - r0);
    uint32_t w[U][4];
    const auto load = [&](int row) {
        const bool live = row < count;
        const uint16_t *p = a.x + (r0 + (live ? row : 0)) * a.ldx;
#pragma unroll
        for (int u = 0; u < U; u++) load_vec<WHOLE, PAST>(w[u], p, 8 * (u * T + t), a.cols, live);
    };
    // sum over the row's threads; `s` is written again only after another barrier
    const auto row_sum = [&](float v, float (&s)[RPW][W]) {
        v = wave_sum(v);
        if constexpr (T > 64) {
            if ((t & 63) == 0) s[grp][t >> 6] = v;
            __syncthreads();
            v = 0.f;
#pragma unroll
            for (int i = 0; i < W; i++) v += s[grp][i];
        }
        return v;
    };
    if constexpr (KEEP) load(grp);  // under way while the parameters come
    // past the row's end x, weight and bias are 0, and with them every term of the sums and y
    float wt[KEEP ? U : 1][8], bs[KEEP ? U : 1][8];
    if constexpr (KEEP) {
        load_params<WHOLE, T>(wt, a.weight, a.param_bf16, 8 * t, a.cols, 1.f);
        load_params<WHOLE, T>(bs, a.bias, a.param_bf16, 8 * t, a.cols, 0.f);
    }
    for (int rb = 0; rb < count; rb += RPW) {
        const bool live = rb + grp < count;
        const int64_t row = r0 + rb + grp;
        if constexpr (!KEEP) load(rb + grp);
        float y[U][8];
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int i = 0; i < 8; i++) {
                y[u][i] = (i & 1) ? bf16_hi(w[u][i >> 1]) : bf16_lo(w[u][i >> 1]);
                sum += y[u][i];
            }
        if constexpr (KEEP) load(rb + grp + RPW);
        float mean = 0.f;
        if (!a.rms) {
            mean = row_mean(row_sum(sum, s0), (float)a.cols, rn);
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int n = a.cols - 8 * (u * T + t);
                const float mu = n > 0 ? mean : 0.f;
#pragma unroll
                for (int i = 0; i < 8; i++) y[u][i] = WHOLE || i < n ? y[u][i] - mu : 0.f;
            }
        } else if (T > 64) {
            __syncthreads();  // the other barrier between two uses of s1
        }
        float sq = 0.f;
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int i = 0; i < 8; i++) sq = __builtin_fmaf(y[u][i], y[u][i], sq);
        const float var = row_sum(sq, s1) * rn;
        const float rstd = rsqrt1(var + a.eps);
        if (live && t == 0) {
            if (a.mean && !a.rms) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = 8 * (u * T + t), n = a.cols - c;
            if constexpr (!KEEP) {
                load_params<WHOLE, T>(wt, a.weight, a.param_bf16, c, a.cols, 1.f);
                load_params<WHOLE, T>(bs, a.bias, a.param_bf16, c, a.cols, 0.f);
            }
            const int k = KEEP ? u : 0;
#pragma unroll
            for (int i = 0; i < 8; i++) y[u][i] = __builtin_fmaf(y[u][i] * rstd, wt[k][i], bs[k][i]);
            if constexpr (TO == TO_BF16) {
                if (live) store_vec<WHOLE>(reinterpret_cast<uint16_t *>(a.out) + row * a.ld_out, y[u], c, a.cols);
            } else {
                float am = __builtin_fabsf(y[u][0]);  // NaN if an element is: one instruction for two elements
#pragma unroll
                for (int i = 1; i < 8; i++) am = __builtin_elementwise_maximum(am, __builtin_fabsf(y[u][i]));
                uint32_t m = __float_as_uint(am) & 0x7FFFFFFFu;
                m = TO == TO_BLOCK ? row16_max(m) : quad_max(m);
                uint8_t *q = reinterpret_cast<uint8_t *>(a.out) + row * a.ld_out;
                if constexpr (TO == TO_BLOCK) {
                    float sc, inv;
                    bool ok;
                    block_scale<F>(m, sc, inv, ok);
                    const uint32_t lo = block_cvt4<F>(y[u][0], y[u][1], y[u][2], y[u][3], inv, ok);
                    const uint32_t hi = block_cvt4<F>(y[u][4], y[u][5], y[u][6], y[u][7], inv, ok);
                    if (live && n > 0) {
                        if (WHOLE) {
                            const uint32_t v[2] = {lo, hi};
                            __builtin_memcpy(q + (uint32_t)c, v, 8);
                        } else {
                            store8(q + (uint32_t)c, lo, hi, n);
                        }
                        if ((t & 15) == 0) sSc[(c / kBlk) * kNormRows + rb + grp] = sc;
                    }
                } else {
                    const bool ok = m < 0x7F800000u;
                    const int e = scale_exp_f32<F>(ok ? m : 0u);
                    const float sc = __builtin_amdgcn_ldexpf(1.0f, e);
                    if (live && n > 0) {  // cols is a multiple of 32: whole vectors
                        if constexpr (F == E2M1) {
                            const uint32_t v = ok ? cvt8_fp4(y[u], sc) : 0u;
                            __builtin_memcpy(q + (uint32_t)(c / 2), &v, 4);
                        } else {
                            const float lim = __builtin_amdgcn_ldexpf(MaxNormal<F>::v, e);
                            const uint32_t v[2] = {ok ? cvt4_fp8<F>(y[u][0], y[u][1], y[u][2], y[u][3], sc, lim) : 0u,
                                                   ok ? cvt4_fp8<F>(y[u][4], y[u][5], y[u][6], y[u][7], sc, lim) : 0u};
                            __builtin_memcpy(q + (uint32_t)c, v, 8);
                        }
                        if ((t & 3) == 0)
                            reinterpret_cast<uint8_t *>(a.scales)[row * a.ld_scales + c / 32] = (uint8_t)(ok ? e + 127 : 0xFF);
                    }
                }
            }
        }
    }
    if constexpr (TO == TO_BLOCK) {
        __syncthreads();
        const int nb = (a.cols + kBlk - 1) / kBlk;
        for (int i = threadIdx.x; i < nb * kNormRows; i += NT) {
            const int b = i / kNormRows, r = i % kNormRows;
            if (r < count) reinterpret_cast<float *>(a.scales)[b * a.ld_scales + r0 + r] = sSc[i];
        }
    }
}

template <int T, int U, int TO, int F>
hipError_t launch_norm_tu(const NormArgs &a, hipStream_t s) {
    constexpr int NT = T < 256 ? 256 : T, RPW = NT / T;
    // rows per workgroup: as many as leave eight workgroups' worth of threads per CU, RPW at least
    const int64_t fill = 256 * 2048 / NT;
    int64_t per = a.rows / fill / RPW * RPW;
    per = per < RPW ? RPW : per > kNormRows ? kNormRows : per;
    const dim3 grid((unsigned)((a.rows + per - 1) / per)), block(NT);
    if (a.cols % 8 != 0) hipLaunchKernelGGL((k_norm<T, U, TO, F, false, false>), grid, block, 0, s, a, (int)per);
    else if (past_cache(a.rows, a.cols)) hipLaunchKernelGGL((k_norm<T, U, TO, F, true, true>), grid, block, 0, s, a, (int)per);
    else hipLaunchKernelGGL((k_norm<T, U, TO, F, true, false>), grid, block, 0, s, a, (int)per);
    return hipGetLastError();
}

template <int TO, int F>
hipError_t launch_norm_to(const NormArgs &a, hipStream_t s) {
    if (a.cols <= 512) return launch_norm_tu<64, 1, TO, F>(a, s);
    if (a.cols <= 1024) return launch_norm_tu<64, 2, TO, F>(a, s);
    if (a.cols <= 2048) return launch_norm_tu<256, 1, TO, F>(a, s);
    if (a.cols <= 4096) return launch_norm_tu<256, 2, TO, F>(a, s);
    if (a.cols <= 8192) return launch_norm_tu<512, 2, TO, F>(a, s);
    if (a.cols <= 16384) return launch_norm_tu<1024, 2, TO, F>(a, s);
    return launch_norm_tu<1024, 4, TO, F>(a, s);
}

// ---------------------------------------------------------------------------
// T threads and 8 T U >= cols elements per row, R rows at a time; workgroup b takes rows
// [b, b + 1) * per.  PARAMS: the sums of dy * xh and dy over those rows go to ws[b][0 and 1][cols].
// Without, R is 1 and rows are read where the loop meets them.
template <int T, int U, int R, bool PARAMS, bool WHOLE, bool PAST>
__global__ __launch_bounds__(T *R) void k_norm_bwd(NormBwdArgs a, int per) {
    constexpr int W = T / 64;
    __shared__ float s0[R][W], s1[R][W];
    __shared__ __attribute__((aligned(16))) float sP[PARAMS && R > 1 ? (R - 1) * T * 16 : 4];
    // a wave's lanes share their row: with its number in a scalar register rows are scalar addresses
    const int t = threadIdx.x % T, grp = __builtin_amdgcn_readfirstlane(threadIdx.x / T);
    const float rn = 1.0f / (float)a.cols;
    const int64_t r0 = (int64_t)blockIdx.x * per;
    const int count = (int)min((int64_t)per, a.rows - r0);  // rows of this workgroup, numbered from 0 below
    uint32_t wx[U][4], wd[U][4];
    float rstd = 0.f, mean = 0.f;
    const auto load = [&](int row) {
        const bool live = row < count;
        const int64_t r = r0 + (live ? row : 0);
#pragma unroll
        for (int u = 0; u < U; u++) {
            load_vec<WHOLE, PAST>(wx[u], a.x + r * a.ldx, 8 * (u * T + t), a.cols, live);
            load_vec<WHOLE, PAST>(wd[u], a.dy + r * a.lddy, 8 * (u * T + t), a.cols, live);
        }
        rstd = a.rstd[r];
        mean = a.rms ? 0.f : a.mean[r];
    };
    const auto get = [](const uint32_t(&w)[4], int i) { return (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); };
    load(grp);  // under way while the weight comes
    float wt[U][8];
    load_params<WHOLE, T>(wt, a.weight, a.param_bf16, 8 * t, a.cols, 1.f);
    float dw[PARAMS ? U : 1][8], db[PARAMS ? U : 1][8];
    if constexpr (PARAMS) {
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int i = 0; i < 8; i++) dw[u][i] = db[u][i] = 0.f;
    }
    for (int rb = 0; rb < count; rb += R) {
        const int row = rb + grp;
        uint32_t cx[U][4], cd[U][4];
        // a row that is not there has x, mean and rstd 0, and with them xh
        const float rs = row < count ? rstd : 0.f, mn = row < count ? mean : 0.f;
        float sg = 0.f, sgx = 0.f;
#pragma unroll
        for (int u = 0; u < U; u++) {
#pragma unroll
            for (int k = 0; k < 4; k++) {
                cx[u][k] = wx[u][k];
                cd[u][k] = wd[u][k];
            }
            // Past the row's end x, dy and g are 0 and x - mean is -mean, and nothing of it may reach the sums over the
            // row: g * rstd comes first, because mean * rstd may be beyond fp32 where no xh is, and 0 * Inf is NaN.
            // (dweight past the end is not stored.)
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float d = get(cd[u], i), xm = get(cx[u], i) - mn, g = d * wt[u][i];
                sg += g;
                sgx = __builtin_fmaf(g * rs, xm, sgx);
                if constexpr (PARAMS) {
                    dw[u][i] = __builtin_fmaf(d, xm * rs, dw[u][i]);
                    db[u][i] += d;
                    // here and now: left alone, the compiler moves these sums to the end of the loop and
                    // holds every d and xh until then
                    asm volatile("" : "+v"(dw[u][i]), "+v"(db[u][i]));
                }
            }
        }
        load(row + R);  // the next rows, under this one's sums and stores
        sg = wave_sum(sg);
        sgx = wave_sum(sgx);
        if constexpr (T > 64) {
            if ((t & 63) == 0) {
                s0[grp][t >> 6] = sg;
                s1[grp][t >> 6] = sgx;
            }
            __syncthreads();
            sg = sgx = 0.f;
#pragma unroll
            for (int i = 0; i < W; i++) {
                sg += s0[grp][i];
                sgx += s1[grp][i];
            }
            __syncthreads();  // the slots are written again for the next rows
        }
        const float mg = a.rms ? 0.f : sg * rn, mgx = sgx * rn;
        // g and xh are made again from the packed values: kept, they would cost 16 U registers (the
        // empty asm keeps the compiler from keeping them)
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = 8 * (u * T + t);
            if (row >= count) continue;
            float d[8];
#pragma unroll
            for (int k = 0; k < 4; k++) asm volatile("" : "+v"(cx[u][k]), "+v"(cd[u][k]));
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float xh = (get(cx[u], i) - mn) * rs, g = get(cd[u], i) * wt[u][i];
                d[i] = __builtin_fmaf(-xh, mgx, g - mg) * rs;
            }
            store_vec<WHOLE>(a.dx + (r0 + row) * a.lddx, d, c, a.cols);
        }
    }
    if constexpr (PARAMS) {
        float *const d = a.ws + (int64_t)blockIdx.x * 2 * a.cols;
#pragma unroll
        for (int u = 0; u < U; u++) {
            if constexpr (R > 1) {  // the R rows' sums meet in group 0
                if (u > 0) __syncthreads();
                if (grp > 0) {
                    float *p = sP + (grp - 1) * T * 16 + t;
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        p[i * T] = dw[u][i];
                        p[(8 + i) * T] = db[u][i];
                    }
                }
                __syncthreads();
                if (grp == 0) {
#pragma unroll 1
                    for (int q = 0; q < R - 1; q++)
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            dw[u][i] += sP[q * T * 16 + t + i * T];
                            db[u][i] += sP[q * T * 16 + t + (8 + i) * T];
                        }
                }
            }
            const int c = 8 * (u * T + t), n = a.cols - c;
            if (grp > 0 || n <= 0) continue;
            const auto put = [&](float *p, const float (&v)[8]) {
                if (n >= 8) {
                    __builtin_memcpy(p, v, 32);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        if (i < n) p[i] = v[i];
                }
            };
            if (a.dw) put(d + c, dw[u]);
            if (a.db) put(d + a.cols + c, db[u]);
        }
    }
}

// Rows wider than that kernel holds: the parameters' sums in a kernel of their own
constexpr int kPartCols = 512;  // columns per workgroup, 8 per lane

// sums of chunk blockIdx.y of the rows: ws[chunk][0 or 1][cols]
__global__ __launch_bounds__(256) void k_norm_dparam(NormBwdArgs a, int64_t per) {
    __shared__ float s[3][2][kPartCols];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * kPartCols + 8 * lane, n = a.cols - c;
    const int64_t r0 = (int64_t)blockIdx.y * per, r1 = min(a.rows, r0 + per);
    float dw[8], db[8];
#pragma unroll
    for (int i = 0; i < 8; i++) dw[i] = db[i] = 0.f;
    if (n > 0) {
        for (int64_t r = r0 + wave; r < r1; r += 4) {
            uint32_t wx[4], wd[4];
            load_vec<false>(wx, a.x + r * a.ldx, c, a.cols, true);
            load_vec<false>(wd, a.dy + r * a.lddy, c, a.cols, true);
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

// the chunks' sums: 64 columns of one of the two gradients per workgroup, sixteen waves taking every
// sixteenth chunk
constexpr int kSumWaves = 16, kSumLoads = 8;
__global__ __launch_bounds__(64 * kSumWaves) void k_norm_dparam_sum(NormBwdArgs a, int chunks) {
    __shared__ float s[kSumWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float *out = blockIdx.y ? a.db : a.dw;
    if (!out) return;  // uniform
    float v = 0.f;
    if (c < a.cols) {
        const float *p = a.ws + (int64_t)blockIdx.y * a.cols + c;
        for (int k = wave; k < chunks; k += kSumLoads * kSumWaves) {
            float t[kSumLoads];  // all under way together, also where they are not of a whole number
#pragma unroll
            for (int i = 0; i < kSumLoads; i++) t[i] = p[(int64_t)min(k + i * kSumWaves, chunks - 1) * 2 * a.cols];
#pragma unroll
            for (int i = 0; i < kSumLoads; i++) v += k + i * kSumWaves < chunks ? t[i] : 0.f;
        }
    }
    s[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && c < a.cols) {
        v = 0.f;
#pragma unroll
        for (int w = 0; w < kSumWaves; w++) v += s[w][lane];
        out[c] = v;
    }
}

// rows of a workgroup at a time (R), and the chunks that the rows are cut into: about one workgroup per CU, and
// none without a row (300 rows: 2 for each of 150 workgroups, not of 256)
int norm_rows_at_once(int64_t cols) {
    return cols <= 2048 ? 8 : cols <= 4096 ? 4 : cols <= 8192 ? 2 : 1;
}
int64_t dparam_chunks(int64_t rows, int64_t cols) {
    if (rows == 0) return 0;
    const int64_t r = cols <= 16384 ? norm_rows_at_once(cols) : 16, n = (rows + r - 1) / r;
    const int64_t most = n < 256 ? n : 256, per = (rows + most - 1) / most;
    return (rows + per - 1) / per;
}

template <int T, int U>
hipError_t launch_dx(const NormBwdArgs &a, hipStream_t s) {
    const int per = (int)((a.rows + (1 << 20) - 1) >> 20);
    const dim3 grid((unsigned)((a.rows + per - 1) / per));
    if (a.cols % 8 != 0) hipLaunchKernelGGL((k_norm_bwd<T, U, 1, false, false, false>), grid, dim3(T), 0, s, a, per);
    else if (past_cache(a.rows, a.cols)) hipLaunchKernelGGL((k_norm_bwd<T, U, 1, false, true, true>), grid, dim3(T), 0, s, a, per);
    else hipLaunchKernelGGL((k_norm_bwd<T, U, 1, false, true, false>), grid, dim3(T), 0, s, a, per);
    return hipGetLastError();
}

template <int T, int U, int R>
hipError_t launch_bwd(const NormBwdArgs &a, int64_t chunks, hipStream_t s) {
    if (!a.dw && !a.db) return launch_dx<T, U>(a, s);
    const int per = (int)((a.rows + chunks - 1) / chunks);
    const dim3 grid((unsigned)chunks), block(T * R);
    if (a.cols % 8 != 0) hipLaunchKernelGGL((k_norm_bwd<T, U, R, true, false, false>), grid, block, 0, s, a, per);
    else if (past_cache(a.rows, a.cols)) hipLaunchKernelGGL((k_norm_bwd<T, U, R, true, true, true>), grid, block, 0, s, a, per);
    else hipLaunchKernelGGL((k_norm_bwd<T, U, R, true, true, false>), grid, block, 0, s, a, per);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs &all, int to, int fmt, hipStream_t s) {
    constexpr int64_t most = (int64_t)1 << 25;  // rows per launch: below 2^32 threads at 1024 for 16 rows
    for (int64_t r = 0; r < all.rows; r += most) {
        NormArgs a = all;
        a.rows = all.rows - r < most ? all.rows - r : most;
        a.x += r * a.ldx;
        a.out = (uint8_t *)a.out + r * a.ld_out * (to == TO_BF16 ? 2 : 1);
        if (to == TO_BLOCK) a.scales = (float *)a.scales + r;
        if (to == TO_MX) a.scales = (uint8_t *)a.scales + r * a.ld_scales;
        if (a.mean) a.mean += r;
        if (a.rstd) a.rstd += r;
        hipError_t e;
        if (to == TO_BF16) e = launch_norm_to<TO_BF16, E4M3>(a, s);
        else if (to == TO_BLOCK) e = fmt == E4M3 ? launch_norm_to<TO_BLOCK, E4M3>(a, s) : launch_norm_to<TO_BLOCK, E5M2>(a, s);
        else if (fmt == E4M3) e = launch_norm_to<TO_MX, E4M3>(a, s);
        else if (fmt == E5M2) e = launch_norm_to<TO_MX, E5M2>(a, s);
        else e = launch_norm_to<TO_MX, E2M1>(a, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

int64_t norm_backward_workspace(int64_t rows, int64_t cols) { return dparam_chunks(rows, cols) * 2 * cols; }

hipError_t launch_norm_backward(const NormBwdArgs &a, hipStream_t s) {
    const bool params = a.dw || a.db;
    const int64_t chunks = dparam_chunks(a.rows, a.cols);
    hipError_t e = hipSuccess;
    if (a.rows > 0) {
        if (a.cols <= 512) e = launch_bwd<64, 1, 8>(a, chunks, s);
        else if (a.cols <= 1024) e = launch_bwd<64, 2, 8>(a, chunks, s);
        else if (a.cols <= 2048) e = launch_bwd<128, 2, 8>(a, chunks, s);
        else if (a.cols <= 4096) e = launch_bwd<256, 2, 4>(a, chunks, s);
        else if (a.cols <= 8192) e = launch_bwd<256, 4, 2>(a, chunks, s);
        else if (a.cols <= 16384) e = launch_bwd<512, 4, 1>(a, chunks, s);
        else {
            e = launch_dx<1024, 4>(a, s);
            if (e == hipSuccess && params) {
                const dim3 grid((unsigned)((a.cols + kPartCols - 1) / kPartCols), (unsigned)chunks);
                hipLaunchKernelGGL(k_norm_dparam, grid, dim3(256), 0, s, a, (a.rows + chunks - 1) / chunks);
                e = hipGetLastError();
            }
        }
    }
    if (e != hipSuccess || !params) return e;
    hipLaunchKernelGGL(k_norm_dparam_sum, dim3((unsigned)((a.cols + 63) / 64), 2), dim3(64 * kSumWaves), 0, s, a,
                       (int)chunks);
    return hipGetLastError();
}

}  // namespace mx
