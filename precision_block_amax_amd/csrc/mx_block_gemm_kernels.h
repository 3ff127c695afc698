// mx_block_gemm_kernels.h -- products of block-128 FP8 operands for gfx950:
//   C[m, n] = sum_b sa[b][m] * sb[b][n] * sum_{k in block b} A[m, k] * B[n, k]
// (B in 128 x 128 tiles: sb[b][n / 128]), both operands with K contiguous.
//
// The scales are arbitrary fp32 numbers, so unlike an MX product this one cannot
// hand them to the matrix instruction: each block's sum P is formed by matrix
// instructions from a zero accumulator and then added, acc += (sa sb) P, by one
// fused multiply-add per element (two where sb differs from column to column).
// Tiles are computed transposed (B's rows as the instruction's rows), so a lane
// holds one row m of C and 16 columns: sa is one value per lane, and with a
// tiled B so is sa * sb.
//
// fp32 output: FP8 codes are converted to bf16 (exact) and multiplied by
// V_MFMA_F32_32X32X16_BF16, whose products are exact and whose sums lose no
// more than fp32 does.  bf16 output: V_MFMA_F32_32X32X64_F8F6F4 on the
// codes themselves, twice the rate.  Measured on gfx950, that instruction adds
// the products of 32 K in a window ending 2^-13 below the largest (the
// unscaled FP8 instructions, 32x32x16 and 16x16x32, do the same): at most 31
// of them lose less than 2^-13 of the largest each, 2^-8 of the block's sum of
// |terms| at the very worst, 30 times below the output's rounding to bf16 on
// data without cancellation.
#pragma once
#include "mx_block_internal.h"
#include "mx_gemm_kernels.h"

namespace mx {
namespace {

// XCD-aware tile order (as tile_of): consecutive workgroups go to the 8 XCDs in
// turn, so each XCD gets a contiguous run of tiles, in groups of 8 tile rows
__device__ __forceinline__ void block_tile_of(const BlockGemmArgs &g, int &tm, int &tn) {
    const int ntiles = g.tiles_m * g.tiles_n;
    const int wg = blockIdx.x, xcd = wg & 7, idx = wg >> 3;
    const int per = ntiles >> 3, rem = ntiles & 7;
    const int lt = xcd * per + (xcd < rem ? xcd : rem) + idx;
    constexpr int GROUP = 8;
    const int group_tiles = GROUP * g.tiles_n;
    const int grp = lt / group_tiles, first = grp * GROUP;
    const int gsz = min(g.tiles_m - first, GROUP), in = lt - grp * group_tiles;
    tm = first + in % gsz;
    tn = in / gsz;
}

// four consecutive columns of row m, starting at n
template <bool BF16OUT>
__device__ __forceinline__ void block_store4(const BlockGemmArgs &g, int m, int n, const float *v) {
    if (m >= g.M) return;
    const int left = g.N - n;
    if constexpr (BF16OUT) {
        uint16_t *p = reinterpret_cast<uint16_t *>(g.c) + (int64_t)m * g.ldc + n;
        const uint32_t t[2] = {bf16x2(v[0], v[1]), bf16x2(v[2], v[3])};
        if (left >= 4) {
            __builtin_memcpy(p, t, 8);
        } else {
            for (int e = 0; e < left; e++) p[e] = (uint16_t)(t[e >> 1] >> (16 * (e & 1)));
        }
    } else {
        float *p = reinterpret_cast<float *>(g.c) + (int64_t)m * g.ldc + n;
        if (left >= 4) {
            __builtin_memcpy(p, v, 16);
        } else {
            for (int e = 0; e < left; e++) p[e] = v[e];
        }
    }
}

// P (32 x 32, transposed) = sum over the 128 K of one block: A row ra, B row rb of the LDS tiles
// (128-byte rows, swizzled), lane half h.  Any order of K will do as long as both operands share
// it: half h takes chunks h, 2 + h, 4 + h, 6 + h.
struct Frag {
    uint4 c[4];
};
__device__ __forceinline__ Frag read_frag(const uint8_t *tile, int row, int h) {
    Frag f;
#pragma unroll
    for (int q = 0; q < 4; q++) f.c[q] = *reinterpret_cast<const uint4 *>(&tile[swz<128>(row, 2 * q + h)]);
    return f;
}

template <int FA, int FB>
__device__ __forceinline__ v16f block_fp8(const Frag &a, const Frag &b) {
    v16f p = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 2; s++) {
        const uint4 x = a.c[2 * s], y = a.c[2 * s + 1], u = b.c[2 * s], v = b.c[2 * s + 1];
        p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            v8i{(int)u.x, (int)u.y, (int)u.z, (int)u.w, (int)v.x, (int)v.y, (int)v.z, (int)v.w},
            v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w}, p, FB, FA, 0, 0, 0, 0);
    }
    return p;
}

struct Frag16 {
    v8bf v[8];
};
template <int F>
__device__ __forceinline__ Frag16 to_bf16(const Frag &f) {
    Frag16 o;
#pragma unroll
    for (int q = 0; q < 4; q++) {
        o.v[2 * q] = to_bf16x8<F>(f.c[q].x, f.c[q].y, 1.0f);
        o.v[2 * q + 1] = to_bf16x8<F>(f.c[q].z, f.c[q].w, 1.0f);
    }
    return o;
}
__device__ __forceinline__ v16f block_bf16(const Frag16 &a, const Frag16 &b) {
    v16f p = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 8; s++) p = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b.v[s], a.v[s], p, 0, 0, 0);
    return p;
}

// ---------------------------------------------------------------------------
// General kernel: any sizes, strides and alignment.  128 x 128 tiles, four
// waves of 64 x 64, codes and scales through registers into LDS, two buffers.
constexpr int GB = 128, GNT = 256;

// 16 bytes at p, n of them valid, the rest 0
__device__ __forceinline__ uint4 load16(const uint8_t *p, int n) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (n >= 16) {
        __builtin_memcpy(&v, p, 16);
    } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 16; i++)
            if (i < n) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
}

template <int FA, int FB, bool BT, bool BF16OUT>
__global__ __launch_bounds__(GNT) void k_block_gemm(BlockGemmArgs g) {
    __shared__ __attribute__((aligned(16))) uint8_t sA[2][GB * kBlk], sB[2][GB * kBlk];
    __shared__ __attribute__((aligned(16))) float sS[2][2 * GB];  // A's rows, B's rows
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1, l32 = lane & 31, h = lane >> 5;
    int tm, tn;
    block_tile_of(g, tm, tn);
    const int m0 = tm * GB, n0 = tn * GB;
    const int nk = (g.K + kBlk - 1) / kBlk;

    uint4 ra[4], rb[4];
    float rs;
    const auto load = [&](int kt) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int id = tid + GNT * i, row = id >> 3, k = kt * kBlk + (id & 7) * 16;
            ra[i] = load16(g.a + (int64_t)min(m0 + row, g.M - 1) * g.lda + k, g.K - k);
            rb[i] = load16(g.b + (int64_t)min(n0 + row, g.N - 1) * g.ldb + k, g.K - k);
        }
        const int r = tid & (GB - 1);
        if (tid < GB) {
            rs = g.as[kt * g.ldsa + min(m0 + r, g.M - 1)];
        } else {
            const int n = min(n0 + r, g.N - 1);
            rs = g.bs[kt * g.ldsb + (BT ? n / kBlk : n)];
        }
    };
    const auto store = [&](int b) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int id = tid + GNT * i, row = id >> 3, ch = id & 7;
            *reinterpret_cast<uint4 *>(&sA[b][swz<128>(row, ch)]) = ra[i];
            *reinterpret_cast<uint4 *>(&sB[b][swz<128>(row, ch)]) = rb[i];
        }
        sS[b][tid] = rs;
    };

    float acc[2][2][16];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[i][j][r] = 0.f;

    load(0);
    store(0);
    __syncthreads();
    for (int kt = 0; kt < nk; kt++) {
        const int b = kt & 1;
        if (kt + 1 < nk) load(kt + 1);
        const float *ss = sS[b];
        Frag fb[2];
        Frag16 gb[2];
#pragma unroll
        for (int j = 0; j < 2; j++) {
            fb[j] = read_frag(sB[b], wn * 64 + j * 32 + l32, h);
            if constexpr (!BF16OUT) gb[j] = to_bf16<FB>(fb[j]);
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const Frag fa = read_frag(sA[b], wm * 64 + i * 32 + l32, h);
            Frag16 ga;
            if constexpr (!BF16OUT) ga = to_bf16<FA>(fa);
            const float sa = ss[wm * 64 + i * 32 + l32];
#pragma unroll
            for (int j = 0; j < 2; j++) {
                v16f p;
                if constexpr (BF16OUT) p = block_fp8<FA, FB>(fa, fb[j]);
                else p = block_bf16(ga, gb[j]);
                if constexpr (BT) {
                    const float s = sa * ss[GB + wn * 64];
#pragma unroll
                    for (int r = 0; r < 16; r++) acc[i][j][r] = __builtin_fmaf(p[r], s, acc[i][j][r]);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const float4 sb = *reinterpret_cast<const float4 *>(&ss[GB + wn * 64 + j * 32 + 8 * q + 4 * h]);
                        const float s4[4] = {sb.x, sb.y, sb.z, sb.w};
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            acc[i][j][4 * q + e] = __builtin_fmaf(p[4 * q + e], sa * s4[e], acc[i][j][4 * q + e]);
                    }
                }
            }
        }
        if (kt + 1 < nk) store(b ^ 1);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int q = 0; q < 4; q++)
                block_store4<BF16OUT>(g, m0 + wm * 64 + i * 32 + l32, n0 + wn * 64 + j * 32 + 8 * q + 4 * h, &acc[i][j][4 * q]);
}

template <int FA, int FB, bool BT, bool BF16OUT>
hipError_t launch_block_gemm_as(BlockGemmArgs g, hipStream_t s) {
    g.tiles_m = (g.M + GB - 1) / GB;
    g.tiles_n = (g.N + GB - 1) / GB;
    hipLaunchKernelGGL((k_block_gemm<FA, FB, BT, BF16OUT>), dim3((unsigned)(g.tiles_m * g.tiles_n)), dim3(GNT), 0, s, g);
    return hipGetLastError();
}

template <int FA, int FB>
hipError_t launch_block_gemm_fmt(const BlockGemmArgs &g, bool bt, bool bf16, hipStream_t s) {
    if (bt) return bf16 ? launch_block_gemm_as<FA, FB, true, true>(g, s) : launch_block_gemm_as<FA, FB, true, false>(g, s);
    return bf16 ? launch_block_gemm_as<FA, FB, false, true>(g, s) : launch_block_gemm_as<FA, FB, false, false>(g, s);
}

}  // namespace
}  // namespace mx
