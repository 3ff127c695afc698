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
// Sums in fp32 (FP8SUMS = false; C in fp32 or bf16): FP8 codes are converted to fp16 (exact) and multiplied by
// V_MFMA_F32_32X32X16_F16, whose products are exact and whose sums lose no
// more than fp32 does (measured: 448 x 448 at any place among 127 equal terms from
// 2^-9 to 2^-5, a block's sum is off by 10 * 2^-24 of its terms at most, where 127
// roundings could cost 127).  FP8SUMS (C in bf16): V_MFMA_F32_32X32X64_F8F6F4
// on the codes themselves, twice the rate.  Measured on gfx950, that instruction adds
// the products of 32 K in a window ending 2^-13 below the largest (the
// unscaled FP8 instructions, 32x32x16 and 16x16x32, do the same): at most 31
// of them lose less than 2^-13 of the largest each, 2^-8 of the block's sum of
// |terms| at the very worst, 30 times below the output's rounding to bf16 on
// data without cancellation.  Both to bf16, FP8 and fp32 sums: 8192 x 6144 x 4096
// 187 and 367 us, 1000 x 4096 x 28672 157 and 225, 48 x 4096 x 14336 16.0 and 16.9.
#pragma once
#include "mx_block_internal.h"
#include "mx_gemm_kernels.h"

namespace mx {
namespace {

// four consecutive columns of row m, starting at n
template <bool FP8SUMS>
__device__ __forceinline__ void block_store4(const BlockGemmArgs &g, int m, int n, const float *v) {
    if (m >= g.M) return;
    const int left = g.N - n;
    if (FP8SUMS || g.c_bf16) {
        uint16_t *p = reinterpret_cast<uint16_t *>(g.c) + (int64_t)m * g.ldc + n;
        const uint32_t t[2] = {bf16x2(v[0], v[1]), bf16x2(v[2], v[3])};
        if (left >= 4) {
            __builtin_memcpy(p, t, 8);
        } else {
#pragma unroll
            for (int e = 0; e < 3; e++)
                if (e < left) p[e] = (uint16_t)(t[e >> 1] >> (16 * (e & 1)));
        }
    } else {
        float *p = reinterpret_cast<float *>(g.c) + (int64_t)m * g.ldc + n;
        if (left >= 4) {
            __builtin_memcpy(p, v, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 3; e++)  // constant indices: v is in registers
                if (e < left) p[e] = v[e];
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

typedef float v4f __attribute__((ext_vector_type(4)));
// 8 codes (lo: 0 .. 3, hi: 4 .. 7) as fp16, exact: E5M2 is the upper byte of an fp16 (one byte permute for
// two codes, half the time of a conversion instruction), E4M3 lies within fp16's range, subnormals too
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
template <int F>
__device__ __forceinline__ v8h to_f16x8(uint32_t lo, uint32_t hi) {
    uint32_t w[4];
    if constexpr (F == E5M2) {
        w[0] = __builtin_amdgcn_perm(0u, lo, 0x010C000Cu);
        w[1] = __builtin_amdgcn_perm(0u, lo, 0x030C020Cu);
        w[2] = __builtin_amdgcn_perm(0u, hi, 0x010C000Cu);
        w[3] = __builtin_amdgcn_perm(0u, hi, 0x030C020Cu);
    } else {
        w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
        w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
        w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
        w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
    }
    return __builtin_bit_cast(v8h, make_uint4(w[0], w[1], w[2], w[3]));
}

struct Frag16 {
    v8h v[8];
};
template <int F>
__device__ __forceinline__ Frag16 to_f16(const Frag &f) {
    Frag16 o;
#pragma unroll
    for (int q = 0; q < 4; q++) {
        o.v[2 * q] = to_f16x8<F>(f.c[q].x, f.c[q].y);
        o.v[2 * q + 1] = to_f16x8<F>(f.c[q].z, f.c[q].w);
    }
    return o;
}
__device__ __forceinline__ v16f block_f16(const Frag16 &a, const Frag16 &b) {
    v16f p = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 8; s++) p = __builtin_amdgcn_mfma_f32_32x32x16_f16(b.v[s], a.v[s], p, 0, 0, 0);
    return p;
}

// the first n bytes of v, the rest 0
__device__ __forceinline__ uint4 keep_bytes(uint4 v, int n) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int d = 0; d < 4; d++) {
        const int k = n - 4 * d;
        w[d] = k >= 4 ? w[d] : k <= 0 ? 0u : w[d] & ((1u << (8 * k)) - 1u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------------------
// General kernel: any sizes, strides and alignment.  128 x 128 tiles, four
// waves of 64 x 64, codes and scales through registers into LDS, two buffers.
// 8192 x 6144 x 4096 with rows of 4104 bytes: bf16 275 us (192 on the pipelined
// kernel with aligned rows), fp32 660 (414).
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

template <int FA, int FB, bool BT, bool FP8SUMS>
__global__ __launch_bounds__(GNT, FP8SUMS ? 2 : 1) void k_block_gemm(BlockGemmArgs g) {
    __shared__ __attribute__((aligned(16))) uint8_t sA[2][GB * kBlk], sB[2][GB * kBlk];
    __shared__ __attribute__((aligned(16))) float sS[2][2 * GB];  // A's rows, B's rows
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1, l32 = lane & 31, h = lane >> 5;
    int tm, tn;
    tile_index(g.tiles_m, g.tiles_n, tm, tn);
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
        static_for<0, 2>([&](auto jj) {
            constexpr int j = decltype(jj)::value;
            fb[j] = read_frag(sB[b], wn * 64 + j * 32 + l32, h);
            if constexpr (!FP8SUMS) gb[j] = to_f16<FB>(fb[j]);
        });
        static_for<0, 4>([&](auto tt) {
            constexpr int i = decltype(tt)::value / 2, j = decltype(tt)::value % 2;
            const Frag fa = read_frag(sA[b], wm * 64 + i * 32 + l32, h);
            const float sa = ss[wm * 64 + i * 32 + l32];
            v16f p;
            if constexpr (FP8SUMS) p = block_fp8<FA, FB>(fa, fb[j]);
            else p = block_f16(to_f16<FA>(fa), gb[j]);
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
        });
        if (kt + 1 < nk) store(b ^ 1);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int q = 0; q < 4; q++)
                block_store4<FP8SUMS>(g, m0 + wm * 64 + i * 32 + l32, n0 + wn * 64 + j * 32 + 8 * q + 4 * h, &acc[i][j][4 * q]);
}

// ---------------------------------------------------------------------------
// Pipelined kernel: codes and scales straight to LDS, two stages of 128 K, one
// of them in flight.
//
// WM x WN waves, each TI x 2 tiles of 32 x 32.  Within a stage the tiles follow
// one another so that the matrix pipe never waits for the vector one: tile t's
// instructions go out, and while they run, tile t - 1's sum is added to its
// accumulators (16 multiply-adds, 64 clocks beside 128 of FP8 matrix work) and
// the next row of A fragments is read from LDS (and, for fp32 sums,
// converted).  The last tile's sum is added in the next stage.
//
// 8192 x 6144 x 4096 with FP8 sums, 256 x 256 tiles: 187 us, 2.2 PFLOP/s, the matrix
// pipe busy 55% of the time at 1.9 GHz; without the loads 140, without the sums'
// additions 171, without the matrix instructions 120, so no one of them bounds
// it.  6144 x 4096 x 8192 to fp32, 256 x 128 tiles: 395 us, 1.04 PFLOP/s, bound by
// the vector pipe: 302 instructions per wave and stage (128 of them conversions,
// 128 additions of sums) beside 1024 clocks of matrix work; without the latter
// it takes as long.  1000 x 4096 x 28672, 128 x 128 tiles, one per CU: 152 us,
// bound by the latency of one stage in flight (128 with operands that L2 holds).
__device__ __forceinline__ void dma4(pipe::v4i r, void *lds, int voff, int soff) {
    // one dword per lane to LDS, as pipe::dma16: lane l lands at lds + 4 l
    const uint32_t m = (uint32_t)(uintptr_t)(pipe::lds_t)lds;
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dword %0, %2, %3 offen lds"
                 :
                 : "v"(voff), "s"(m), "s"(r), "s"(soff)
                 : "memory", "m0");
}

constexpr int kDead = (int)0x80000000u;  // a lane offset beyond every buffer: the load writes zeros

// Configurations: tiles per wave, waves.  KG groups of waves take every KG-th stage each, with
// rings of their own, and their sums meet at the end: a 128 x 128 tile has work for four waves of 64 x 64
// only, and a SIMD with one wave neither multiplies while it reads LDS nor the other way round.
// PF: prefetch into L2 (below).
struct Cfg256x256 { static constexpr int TI = 4, WM = 2, WN = 4, KG = 1; static constexpr bool PF = false; };
struct Cfg256x128 { static constexpr int TI = 2, WM = 4, WN = 2, KG = 1; static constexpr bool PF = false; };
struct Cfg128x128 { static constexpr int TI = 2, WM = 2, WN = 2, KG = 2; static constexpr bool PF = false; };
struct Cfg128x128Far : Cfg128x128 { static constexpr bool PF = true; };

// RAG: K ends inside a chunk of 16 bytes.  The stages leave that chunk out, and its products are added after them
// from registers (a branch for it in the loop made the compiler spill: up to 200 registers).  256 x 256 tiles spill
// 48 registers there, 24 instructions after the loop and none in it: 8192 x 6144 x 4095 to bf16 217 us beside 194 of
// 4096; 4104 238, rows of 4112 bytes, whose 128 of a stage lie in two lines.
template <int FA, int FB, bool BT, bool FP8SUMS, class CFG, bool RAG>
__global__ __launch_bounds__(64 * CFG::WM * CFG::WN * CFG::KG, CFG::WM * CFG::WN * CFG::KG / 4) void k_block_gemm_pipe(BlockGemmArgs g) {
    constexpr int TI = CFG::TI, WM = CFG::WM, WN = CFG::WN, NS = 2, KG = CFG::KG;
    static_assert(KG == 1 || (KG == 2 && TI == 2), "the join swaps two rows of tiles");
    constexpr int NW = WM * WN, PM = WM * TI * 32, PN = WN * 64;
    constexpr int NIA = PM / 8 / NW, NIB = PN / 8 / NW;  // 1 KiB loads (8 rows) per wave and stage
    static_assert(NIA >= 1 && NIB >= 1 && PM % (8 * NW) == 0 && PN % (8 * NW) == 0, "load split");
    static_assert((PM + PN) / 64 <= NW, "one scale load per wave");
    constexpr bool PF = CFG::PF;
    constexpr int ST = (PM + PN) * kBlk, SR = 2 * NS;
    // A's stages of codes, then B's: a fragment read is one of eight lane offsets (four 32-byte
    // steps of K, two operands), the stage's place and a constant
    constexpr int OB = NS * PM * kBlk;
    __shared__ __attribute__((aligned(16))) uint8_t sCodes[KG * NS * ST];
    // scales, in a ring of their own: the last tile of a stage is scaled in the next one, while the
    // loads that reuse the stage's codes are under way
    __shared__ __attribute__((aligned(16))) float sScales[KG * SR * (PM + PN)];
    __shared__ uint32_t sDump[PF ? 64 : 1];  // where the prefetches' words go
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave_all = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int grp = KG == 1 ? 0 : wave_all / NW, wave = wave_all % NW;
    uint8_t *const sC = sCodes + grp * NS * ST;
    float *const sS = sScales + grp * SR * (PM + PN);
    const int wm = wave / WN, wn = wave % WN, l32 = lane & 31, h = lane >> 5;
    int tm, tn;
    tile_index(g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * PM, n0 = tn * PN;
    const int K = RAG ? g.K & ~15 : g.K, nk = (K + kBlk - 1) / kBlk, ktail = K - (nk - 1) * kBlk;
    const int mrows = min(PM, g.M - m0), nrows = min(PN, g.N - n0);
    const int lda = (int)g.lda, ldb = (int)g.ldb;
    // rows past the operand lie past its records, whichever part of the offset is the scalar one (the range check
    // counts both: measured), and read as zeros
    const pipe::v4i rA = pipe::rsrc(g.a + (int64_t)m0 * lda, (uint32_t)mrows * lda);
    const pipe::v4i rB = pipe::rsrc(g.b + (int64_t)n0 * ldb, (uint32_t)nrows * ldb);

    // lane l of a load fills 16-byte slot l % 8 of row l / 8 of its 8 rows, i.e. logical chunk
    // (l % 8) ^ key(row); the key of the rows of odd loads differs in bit 2.  In K's last stage
    // the chunks past K are dead, in a stage past it all are.
    const int rowA = wave * NIA * 8 + lane / 8, rowB = wave * NIB * 8 + lane / 8;
    int vA[2], vB[2];
    bool inA[2], inB[2];  // the chunk lies before the end of K in the last stage
#pragma unroll
    for (int o = 0; o < 2; o++) {
        const int ca = ((lane & 7) ^ swz_key<128>(rowA + 8 * o)) << 4, cb = ((lane & 7) ^ swz_key<128>(rowB + 8 * o)) << 4;
        vA[o] = rowA * lda + ca;
        vB[o] = rowB * ldb + cb;
        inA[o] = ca < ktail;
        inB[o] = cb < ktail;
    }
    // scales: wave w < PM / 64 loads those of A's rows 64 w .., the next PN / 64 waves those of B's rows
    // (waves beyond repeat them)
    constexpr int WA = PM / 64, WB = PN / 64;
    const bool isA = wave < WA;
    const int sw = isA ? wave : (wave - WA) % WB;
    const float *sbase = isA ? g.as + m0 : g.bs + (BT ? n0 / kBlk : n0);
    const int64_t lds_ = isA ? g.ldsa : g.ldsb;
    const int swidth = isA ? mrows : (BT ? (nrows + kBlk - 1) / kBlk : nrows);
    const pipe::v4i rS = pipe::rsrc(sbase, (uint32_t)(((int64_t)(nk - 1) * lds_ + swidth) * 4));
    const int srow = 64 * sw + lane;
    const int vS = (isA || !BT ? srow : srow / kBlk) * 4;
    float *const sdst = sS + (isA ? 0 : PM) + 64 * sw;

    // Prefetch into L2.  A stage takes 128 bytes of each row, rows far apart; operands that come from beyond
    // the last-level cache then open a DRAM page for every one of them, and a stage's loads wait for its
    // slowest.  One wave of either group fetches a word of every line of whole KiB of rows, the next KiB of
    // K, a few rows per stage: the first group A's rows, the second B's.  The 32 tiles that an XCD works on
    // are 8 x 4 (tile_index), so a workgroup takes a quarter of its A rows and an eighth of its B rows; with
    // fewer than eight rows of tiles the eighths of B that would be theirs are not fetched ahead.
    // Operands from HBM, without and with: 1000 x 4096 x 28672 180 and 155 us, 512 x 8192 x 28672 (four rows of
    // tiles) 188 and 177, 256 x 16384 x 28672 (two) 200 and 193.  1000 rows, two or four KiB ahead 166, 168; a line
    // per row and stage, three stages ahead, 168.
    static_assert(!PF || KG == 2, "a group for each operand");
    constexpr int PW = 8 / KG;  // stages of a group per KiB
    const bool pw = PF && wave == 0;
    const int pper = (grp ? PN / 8 : PM / 4) / PW, pbase = grp ? (tm & 7) * (PN / 8) : (tn & 3) * (PM / 4);
    const int prow0 = pbase + lane / 8, plim = lane / 8 < pper ? (grp ? nrows : mrows) : 0, pld = grp ? ldb : lda;
    const pipe::v4i rP = grp ? rB : rA;

    const auto issue = [&](int u, int it) {  // the group's stage number `it` into place u
        const int kt = it * KG + grp;
        const bool live = kt < nk, last = kt == nk - 1;
        const int so = live ? kt * kBlk : 0;
        uint8_t *const dA = sC + u * PM * kBlk + wave * NIA * 1024, *const dB = sC + OB + u * PN * kBlk + wave * NIB * 1024;
        int a[2], b[2];
#pragma unroll
        for (int o = 0; o < 2; o++) {
            a[o] = live && (!last || inA[o]) ? vA[o] : kDead;
            b[o] = live && (!last || inB[o]) ? vB[o] : kDead;
        }
#pragma unroll
        for (int q = 0; q < NIA; q++) pipe::dma16(rA, dA + q * 1024, a[q & 1], so + q * 8 * lda);
#pragma unroll
        for (int q = 0; q < NIB; q++) pipe::dma16(rB, dB + q * 1024, b[q & 1], so + q * 8 * ldb);
        dma4(rS, sdst + (it & (SR - 1)) * (PM + PN), live ? vS : kDead, live ? kt * (int)lds_ * 4 : 0);
        if constexpr (PF) {
            const int pr = prow0 + it % PW * pper, pk = (it / PW + 1) * 1024 + (lane & 7) * 128;
            dma4(rP, sDump, pw && pr < plim && pk < K ? pr * pld + pk : kDead, 0);
        }
    };

    float acc[TI][2][16];
#pragma unroll
    for (int i = 0; i < TI; i++)
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[i][j][r] = 0.f;

    v16f pp = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};  // sum of the tile before
    float ps = 0.f;                                                                                // its scale (A's, without BT)
    const int scol = PM + wn * 64 + (BT ? 0 : 4 * h);
    // without BT: the scales of its columns.  There is no tile before the first: its sum is 0 and so
    // are its scales, in the place that the ring fills last.
    const float *psb = sS + (SR - 1) * (PM + PN) + scol;
    if constexpr (!BT) {
        for (int i = tid % (64 * NW); i < PN; i += 64 * NW) sS[(SR - 1) * (PM + PN) + PM + i] = 0.f;
    }
    // acc += scale * sum of the tile before
    const auto promote = [&](float (&c)[16], const float4 (&sb)[4]) {
        if constexpr (BT) {
#pragma unroll
            for (int r = 0; r < 16; r++) c[r] = __builtin_fmaf(pp[r], ps, c[r]);
        } else {
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const float s4[4] = {sb[q].x, sb[q].y, sb[q].z, sb[q].w};
#pragma unroll
                for (int e = 0; e < 4; e++) c[4 * q + e] = __builtin_fmaf(pp[4 * q + e], ps * s4[e], c[4 * q + e]);
            }
        }
    };
    const auto read_sb = [&](float4 (&sb)[4]) {
        if constexpr (!BT) {
#pragma unroll
            for (int q = 0; q < 4; q++) sb[q] = *reinterpret_cast<const float4 *>(psb + 8 * q);
        }
    };

    // lane offsets of the fragments' chunks 2 q + h; rows 32 apart share the key
    const uint8_t *pa[4], *pb[4];
#pragma unroll
    for (int q = 0; q < 4; q++) {
        const int ch = ((2 * q + h) ^ swz_key<128>(l32)) << 4;
        pa[q] = sC + (wm * TI * 32 + l32) * kBlk + ch;
        pb[q] = sC + OB + (wn * 64 + l32) * kBlk + ch;
    }
    const auto frag = [](const uint8_t *const (&p)[4], int off) {
        Frag f;
#pragma unroll
        for (int q = 0; q < 4; q++) f.c[q] = *reinterpret_cast<const uint4 *>(p[q] + off);
        return f;
    };

    // Stage `it` of the group, in place u, has landed for every wave, and every wave is done with the reads of
    // the stage before it, whose place takes the stage after it.
    const auto arrive = [&](int u, int it) {
        pipe::wait_vm<PF>();  // the youngest load is a prefetch
        pipe::barrier();
        issue(u ^ 1, it + 1);
    };

    // EARLY: a stage begins with its first fragments in registers.  All its LDS reads are out before its
    // last two tiles, so the next stage arrives there: the barrier, the loads' issue and the next stage's
    // first reads fall into those tiles' matrix work instead of standing between two stages.  fp32 sums,
    // 6144 x 4096 x 8192: 400 -> 381 us.  FP8 sums have no registers left for it in 256 x 256 tiles (13
    // spilled: 187 -> 210 us) and gain nothing in 128 x 128 (47.7, 48.9 us).
    constexpr bool EARLY = !FP8SUMS;
    Frag fa[2], fb[2];
    const auto stage = [&](int u, int it) {
        const float *const ss = sS + (it & (SR - 1)) * (PM + PN);
        const int ua = u * PM * kBlk, ub = u * PN * kBlk;
        Frag16 ga, gb[2];
        if constexpr (!EARLY) {
            arrive(u, it);
            fa[0] = frag(pa, ua);
            fb[0] = frag(pb, ub);
        }
        fb[1] = frag(pb, ub + 32 * kBlk);
        float sa[TI];
#pragma unroll
        for (int i = 0; i < TI; i++) sa[i] = ss[wm * TI * 32 + i * 32 + l32];
        const float sbt = BT ? ss[scol] : 1.0f;
        if constexpr (!FP8SUMS) {
            ga = to_f16<FA>(fa[0]);
#pragma unroll
            for (int j = 0; j < 2; j++) gb[j] = to_f16<FB>(fb[j]);
        }
        static_for<0, 2 * TI>([&](auto tt) {
            constexpr int t = decltype(tt)::value, i = t / 2, j = t % 2;
            constexpr int pi = t ? (t - 1) / 2 : TI - 1, pj = t ? (t - 1) % 2 : 1;  // the tile before
            if constexpr (EARLY && t == 2 * TI - 2) arrive(u ^ 1, it + 1);
            if constexpr (j == 0 && i + 1 < TI) fa[(i + 1) & 1] = frag(pa, ua + (i + 1) * 32 * kBlk);
            if constexpr (EARLY && t == 2 * TI - 1) {
                static_assert(TI % 2 == 0, "the last row's fragments are in fa[1]");
                fa[0] = frag(pa, (u ^ 1) * PM * kBlk);
                fb[0] = frag(pb, (u ^ 1) * PN * kBlk);
            }
            float4 sb[4];
            read_sb(sb);
            v16f p;
            if constexpr (FP8SUMS) p = block_fp8<FA, FB>(fa[i & 1], fb[j]);
            else p = block_f16(ga, gb[j]);
            __builtin_amdgcn_sched_barrier(0);
            promote(acc[pi][pj], sb);
            if constexpr (!FP8SUMS && j == 1 && i + 1 < TI) ga = to_f16<FA>(fa[(i + 1) & 1]);
            pp = p;
            ps = BT ? sa[i] * sbt : sa[i];
            psb = ss + scol + j * 32;
            __builtin_amdgcn_sched_barrier(0);
        });
    };

    // two stages at a time, so that their places are constants; past the end of K they are all zeros
    const int nit = (nk + KG - 1) / KG;
    issue(0, 0);
    if constexpr (EARLY) {
        arrive(0, 0);
        fa[0] = frag(pa, 0);
        fb[0] = frag(pb, 0);
    }
    for (int it = 0; it < nit; it += 2) {
        stage(0, it);
        stage(1, it + 1);
    }
    {
        float4 sb[4];
        read_sb(sb);
        promote(acc[TI - 1][1], sb);
    }
    if constexpr (RAG) {
        if (grp == 0) {
            const int kb = K / kBlk;
            const auto chunk = [&](const uint8_t *p) {
                uint4 v;
                __builtin_memcpy(&v, p + K, 16);
                return v;
            };
            const int left = h ? 0 : g.K - K;  // the first half of the lanes holds the chunk, the other one zeros
            uint4 ca[TI];
            float sa[TI];
#pragma unroll
            for (int i = 0; i < TI; i++) {
                const int m = m0 + min((wm * TI + i) * 32 + l32, mrows - 1);
                ca[i] = chunk(g.a + (int64_t)m * lda);
                sa[i] = g.as[kb * g.ldsa + m];
            }
            static_for<0, 2>([&](auto jj) {
                constexpr int j = decltype(jj)::value;
                const int n = wn * 64 + j * 32;
                const uint4 b = keep_bytes(chunk(g.b + (int64_t)(n0 + min(n + l32, nrows - 1)) * ldb), left);
                float sb[16];
                if constexpr (BT) {
                    sb[0] = g.bs[kb * g.ldsb + (n0 + min(n, nrows - 1)) / kBlk];
                } else {
#pragma unroll
                    for (int r = 0; r < 16; r++) sb[r] = g.bs[kb * g.ldsb + n0 + min(n + 8 * (r / 4) + 4 * h + r % 4, nrows - 1)];
                }
                static_for<0, TI>([&](auto ii) {
                    constexpr int i = decltype(ii)::value;
                    __builtin_amdgcn_sched_barrier(0);  // one tile at a time
                    const uint4 a = keep_bytes(ca[i], left);
                    v16f p = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    if constexpr (FP8SUMS) {
                        p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                            v8i{(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0},
                            v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0}, p, FB, FA, 0, 0, 0, 0);
                    } else {
                        p = __builtin_amdgcn_mfma_f32_32x32x16_f16(to_f16x8<FB>(b.x, b.y), to_f16x8<FA>(a.x, a.y), p, 0, 0, 0);
                        p = __builtin_amdgcn_mfma_f32_32x32x16_f16(to_f16x8<FB>(b.z, b.w), to_f16x8<FA>(a.z, a.w), p, 0, 0, 0);
                    }
#pragma unroll
                    for (int r = 0; r < 16; r++) acc[i][j][r] = __builtin_fmaf(p[r], sa[i] * sb[BT ? 0 : r], acc[i][j][r]);
                });
            });
        }
    }
    pipe::wait_vm<0>();
    pipe::barrier();  // every wave has left the loop: the stages' LDS is free

    // two groups: each keeps one row of tiles of every wave's (its own number) and gives the other one
    constexpr int TK = TI / KG;
    if constexpr (KG == 2) {
        float *const mine = reinterpret_cast<float *>(sCodes) + wave_all * 32 * 64;
        const float *const other = reinterpret_cast<const float *>(sCodes) + (wave_all ^ NW) * 32 * 64;
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int r = 0; r < 16; r++) {
                mine[(j * 16 + r) * 64 + lane] = grp ? acc[0][j][r] : acc[1][j][r];
                acc[0][j][r] = grp ? acc[1][j][r] : acc[0][j][r];
            }
        pipe::barrier();
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[0][j][r] += other[(j * 16 + r) * 64 + lane];
        pipe::barrier();
    }

    // C through LDS, each wave its own part, TI2 x 32 rows at a time, so that rows leave as runs of 64
    // elements; 16-byte chunks are XOR-swizzled by the row
    constexpr int ESZ = FP8SUMS ? 2 : 4, ROWB = 64 * ESZ, CPR = ROWB / 16, REG = NS * ST / NW;
    constexpr int TI2 = TK * 32 * ROWB <= REG ? TK : TK / 2;
    static_assert(TI2 >= 1 && TK % TI2 == 0 && TI2 * 32 * ROWB <= REG, "staging");
    uint8_t *const reg = sC + wave * REG;
    const int mbase = m0 + (wm * TI + grp) * 32, nbase = n0 + wn * 64;
    const bool vec = nbase + 64 <= g.N && g.ldc % (16 / ESZ) == 0 && ((uintptr_t)g.c & 15) == 0;
#pragma unroll
    for (int pass = 0; pass < TK / TI2; pass++) {
#pragma unroll
        for (int ii = 0; ii < TI2; ii++) {
            const int m = ii * 32 + l32;
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const float *v = &acc[pass * TI2 + ii][j][4 * q];
                    if constexpr (FP8SUMS)
                        *reinterpret_cast<uint2 *>(&reg[m * ROWB + (((4 * j + q) ^ (m & 7)) << 4) + 8 * h]) =
                            make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
                    else
                        *reinterpret_cast<float4 *>(&reg[m * ROWB + (((8 * j + 2 * q + h) ^ (m & 15)) << 4)]) =
                            make_float4(v[0], v[1], v[2], v[3]);
                }
        }
#pragma unroll
        for (int k = 0; k < TI2 * 32 * CPR / 64; k++) {
            const int m = k * (64 / CPR) + lane / CPR, c = lane % CPR;
            const uint4 t = *reinterpret_cast<const uint4 *>(&reg[m * ROWB + ((c ^ (m & (CPR - 1))) << 4)]);
            const int gm = mbase + pass * TI2 * 32 + m, gn = nbase + c * (16 / ESZ);
            if (gm >= g.M) continue;
            const int64_t at = (int64_t)gm * g.ldc + gn;
            typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
            typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
            if (FP8SUMS || !g.c_bf16) {
                uint8_t *const d = reinterpret_cast<uint8_t *>(g.c) + at * ESZ;
                if (vec) {
                    __builtin_nontemporal_store(u32x4{t.x, t.y, t.z, t.w}, reinterpret_cast<u32x4 *>(d));
                    continue;
                }
                const uint32_t w4[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                for (int e = 0; e < 16 / ESZ; e++) {
                    if (gn + e >= g.N) break;
                    if constexpr (FP8SUMS) reinterpret_cast<uint16_t *>(d)[e] = (uint16_t)(w4[e >> 1] >> (16 * (e & 1)));
                    else reinterpret_cast<uint32_t *>(d)[e] = w4[e];
                }
            } else {  // four sums, rounded to bf16 here
                uint16_t *const d = reinterpret_cast<uint16_t *>(g.c) + at;
                const u32x2 b = {bf16x2(__uint_as_float(t.x), __uint_as_float(t.y)), bf16x2(__uint_as_float(t.z), __uint_as_float(t.w))};
                if (vec) {
                    __builtin_nontemporal_store(b, reinterpret_cast<u32x2 *>(d));
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (gn + e < g.N) d[e] = (uint16_t)(b[e >> 1] >> (16 * (e & 1)));
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Kernel for few rows: tiles of 8 AI x 16 NT of C, a workgroup's eight waves each
// taking every eighth block of K for the whole tile, joined in LDS.
//
// With one row the product is bound by B's bytes.  16 rows of B per workgroup
// make 256 workgroups from N = 4096 on, and the waves' blocks in flight cover
// the latency without a split of K over workgroups, which would need memory to
// join them.  Blocks come straight to LDS, a ring of S per wave and no barrier:
// a fragment's lanes are rows, and loaded into registers its neighbouring lanes
// read different lines, of which an L1 serves one per clock: 48 rows by 4096 x
// 14336 took 28 us at 16 bytes per clock and CU, whatever was in flight; through
// LDS 16 us, 3.7 TB/s of its operands, and 256 times A besides from L2.  1 x 6144 x
// 4096 takes 7.5 us, 3.4 TB/s, of which launch and a first read's latency are half.
constexpr int DW = 8;  // waves

struct Frag2 {
    uint4 c[2];
};

template <int FA, int FB, bool FP8SUMS>
__device__ __forceinline__ v4f few_block(const Frag2 &a, const Frag2 &b) {
    v4f p = {0.f, 0.f, 0.f, 0.f};
    const uint4 x = a.c[0], y = a.c[1], u = b.c[0], v = b.c[1];
    if constexpr (FP8SUMS) {
        p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            v8i{(int)u.x, (int)u.y, (int)u.z, (int)u.w, (int)v.x, (int)v.y, (int)v.z, (int)v.w},
            v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w}, p, FB, FA, 0, 0, 0, 0);
    } else {
        p = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_f16x8<FB>(u.x, u.y), to_f16x8<FA>(x.x, x.y), p, 0, 0, 0);
        p = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_f16x8<FB>(u.z, u.w), to_f16x8<FA>(x.z, x.w), p, 0, 0, 0);
        p = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_f16x8<FB>(v.x, v.y), to_f16x8<FA>(y.x, y.y), p, 0, 0, 0);
        p = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_f16x8<FB>(v.z, v.w), to_f16x8<FA>(y.z, y.w), p, 0, 0, 0);
    }
    return p;
}

// AI: loads of 8 rows of A; with an odd AI the rest of the matrix instruction's 16 rows is whatever LDS
// holds, and reaches only rows of C that do not exist
template <int FA, int FB, bool BT, bool FP8SUMS, int AI, int NT, int S>
__global__ __launch_bounds__(64 * DW) void k_block_gemm_few(BlockGemmArgs g) {
    constexpr int MT = (AI + 1) / 2, DM = 16 * MT, DN = 16 * NT, JP = DN + 4;
    constexpr int OB = MT * 2048, OS = OB + NT * 2048, BLK = OS + 512;  // a block: A's rows, B's, scales of A, of B
    constexpr int LPB = AI + 2 * NT + 2;                                // loads per block
    constexpr int JOIN = DW * DM * JP * 4;                              // the waves' sums
    __shared__ __attribute__((aligned(16))) uint8_t sR[DW * S * BLK > JOIN ? DW * S * BLK : JOIN];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, h = lane >> 4;
    int tm, tn;
    tile_index(g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * 8 * AI, n0 = tn * DN;
    const int nk = (g.K + kBlk - 1) / kBlk, ktail = g.K - (nk - 1) * kBlk;
    const int lda = (int)g.lda, ldb = (int)g.ldb, mrows = min(8 * AI, g.M - m0), nrows = min(DN, g.N - n0);
    // rows end at a multiple of 16 bytes: an aligned 16 bytes that hold a byte of the row
    const int kend = (g.K + 15) & ~15;
    const pipe::v4i rA = pipe::rsrc(g.a + (int64_t)m0 * lda, (uint32_t)((mrows - 1) * lda + kend));
    const pipe::v4i rB = pipe::rsrc(g.b + (int64_t)n0 * ldb, (uint32_t)((nrows - 1) * ldb + kend));
    const pipe::v4i rSA = pipe::rsrc(g.as + m0, (uint32_t)(((int64_t)(nk - 1) * g.ldsa + mrows) * 4));
    const pipe::v4i rSB = pipe::rsrc(g.bs + (BT ? n0 / kBlk : n0), (uint32_t)(((int64_t)(nk - 1) * g.ldsb + (BT ? 1 : nrows)) * 4));
    // lane l of a load: 16-byte slot l % 8 of row l / 8, logical chunk (l % 8) ^ key
    const int lr = lane / 8;
    int vA[AI], vB[2 * NT], cA[2];
#pragma unroll
    for (int o = 0; o < 2; o++) cA[o] = ((lane & 7) ^ swz_key<128>(lr + 8 * o)) << 4;
#pragma unroll
    for (int o = 0; o < 2 * NT; o++) vB[o] = lr + 8 * o < nrows ? (lr + 8 * o) * ldb + cA[o & 1] : kDead;
#pragma unroll
    for (int o = 0; o < AI; o++) vA[o] = lr + 8 * o < mrows ? (lr + 8 * o) * lda + cA[o & 1] : kDead;
    const int vSA = lane < mrows ? lane * 4 : kDead, vSB = BT ? 0 : lane < nrows ? lane * 4 : kDead;
    uint8_t *const ring = sR + wave * S * BLK;

    const auto issue = [&](int slot, int i) {  // block number i of this wave
        const int kt = wave + i * DW;
        const bool live = kt < nk, last = kt == nk - 1;
        uint8_t *const d = ring + slot * BLK;
        const int so = live ? kt * kBlk : 0;
        const bool in[2] = {live && (!last || cA[0] < ktail), live && (!last || cA[1] < ktail)};
#pragma unroll
        for (int o = 0; o < AI; o++) pipe::dma16(rA, d + o * 1024, in[o & 1] ? vA[o] : kDead, so);
#pragma unroll
        for (int o = 0; o < 2 * NT; o++) pipe::dma16(rB, d + OB + o * 1024, in[o & 1] ? vB[o] : kDead, so);
        dma4(rSA, d + OS, live ? vSA : kDead, live ? kt * (int)g.ldsa * 4 : 0);
        dma4(rSB, d + OS + 256, live ? vSB : kDead, live ? kt * (int)g.ldsb * 4 : 0);
    };

    float acc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
            for (int r = 0; r < 4; r++) acc[i][j][r] = 0.f;
    const int count = nk > wave ? (nk - wave + DW - 1) / DW : 0;
    const int ch[2] = {(h ^ swz_key<128>(l16)) << 4, ((4 + h) ^ swz_key<128>(l16)) << 4};  // this lane's chunks: h and 4 + h

#pragma unroll
    for (int i = 0; i < S; i++) issue(i, i);
    int slot = 0;
    for (int i = 0; i < count; i++) {
        pipe::wait_vm<(S - 1) * LPB>();
        // what the loads wrote to LDS is read below: no read may move up past the wait, which the compiler takes for
        // an instruction without effect on memory
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        const uint8_t *const d = ring + slot * BLK;
        Frag2 fa[MT], fb[NT];
        float sa[MT], sb[NT][BT ? 1 : 4];
#pragma unroll
        for (int j = 0; j < NT; j++) {
#pragma unroll
            for (int q = 0; q < 2; q++) fb[j].c[q] = *reinterpret_cast<const uint4 *>(d + OB + (16 * j + l16) * kBlk + ch[q]);
            if constexpr (BT) {
                sb[j][0] = *reinterpret_cast<const float *>(d + OS + 256);
            } else {
                const float4 t = *reinterpret_cast<const float4 *>(d + OS + 256 + 64 * j + 16 * h);
                sb[j][0] = t.x;
                sb[j][1] = t.y;
                sb[j][2] = t.z;
                sb[j][3] = t.w;
            }
        }
#pragma unroll
        for (int t = 0; t < MT; t++) {
#pragma unroll
            for (int q = 0; q < 2; q++) fa[t].c[q] = *reinterpret_cast<const uint4 *>(d + (16 * t + l16) * kBlk + ch[q]);
            sa[t] = *reinterpret_cast<const float *>(d + OS + (16 * t + l16) * 4);
        }
        // the slot's values are in registers before its next block may land
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        issue(slot, i + S);
        slot = slot + 1 == S ? 0 : slot + 1;
        if (wave + i * DW == nk - 1 && ktail % 16 != 0) {  // the row's end inside a chunk
#pragma unroll
            for (int q = 0; q < 2; q++) {
                const int n = ktail - (4 * q + h) * 16;
#pragma unroll
                for (int j = 0; j < NT; j++) fb[j].c[q] = keep_bytes(fb[j].c[q], n);
#pragma unroll
                for (int t = 0; t < MT; t++) fa[t].c[q] = keep_bytes(fa[t].c[q], n);
            }
        }
#pragma unroll
        for (int t = 0; t < MT; t++)
#pragma unroll
            for (int j = 0; j < NT; j++) {
                const v4f p = few_block<FA, FB, FP8SUMS>(fa[t], fb[j]);
#pragma unroll
                for (int r = 0; r < 4; r++) acc[t][j][r] = __builtin_fmaf(p[r], sa[t] * sb[j][BT ? 0 : r], acc[t][j][r]);
            }
    }
    pipe::wait_vm<0>();
    pipe::barrier();  // every wave's blocks are done with: the join may use their LDS

    // lane: row m = l16 of tile (t, j), columns 4 h .. 4 h + 3
    float *const sJ = reinterpret_cast<float *>(sR);
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
        for (int j = 0; j < NT; j++)
            *reinterpret_cast<float4 *>(&sJ[(wave * DM + 16 * t + l16) * JP + 16 * j + 4 * h]) =
                make_float4(acc[t][j][0], acc[t][j][1], acc[t][j][2], acc[t][j][3]);
    __syncthreads();
    for (int i = tid; i < DM * DN / 4; i += 64 * DW) {
        const int m = i / (DN / 4), n = i % (DN / 4) * 4;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < DW; w++) {
            const float4 x = *reinterpret_cast<const float4 *>(&sJ[(w * DM + m) * JP + n]);
            v[0] += x.x;
            v[1] += x.y;
            v[2] += x.z;
            v[3] += x.w;
        }
        if (m < 8 * AI) block_store4<FP8SUMS>(g, m0 + m, n0 + n, v);
    }
}

template <int FA, int FB, bool BT, bool FP8SUMS, int AI, int NT, int S>
hipError_t launch_block_gemm_few(BlockGemmArgs g, hipStream_t s) {
    g.tiles_m = (g.M + 8 * AI - 1) / (8 * AI);
    g.tiles_n = (g.N + 16 * NT - 1) / (16 * NT);
    hipLaunchKernelGGL((k_block_gemm_few<FA, FB, BT, FP8SUMS, AI, NT, S>), dim3((unsigned)(g.tiles_m * g.tiles_n)),
                       dim3(64 * DW), 0, s, g);
    return hipGetLastError();
}

template <int FA, int FB, bool BT, bool FP8SUMS, class CFG, bool RAG>
hipError_t launch_block_gemm_pipe(BlockGemmArgs g, hipStream_t s) {
    constexpr int PM = CFG::WM * CFG::TI * 32, PN = CFG::WN * 64;
    g.tiles_m = (g.M + PM - 1) / PM;
    g.tiles_n = (g.N + PN - 1) / PN;
    hipLaunchKernelGGL((k_block_gemm_pipe<FA, FB, BT, FP8SUMS, CFG, RAG>), dim3((unsigned)(g.tiles_m * g.tiles_n)),
                       dim3(64 * CFG::WM * CFG::WN * CFG::KG), 0, s, g);
    return hipGetLastError();
}

template <int FA, int FB, bool BT, bool FP8SUMS, class CFG>
hipError_t launch_block_gemm_k(const BlockGemmArgs &g, hipStream_t s) {
    return g.K % 16 ? launch_block_gemm_pipe<FA, FB, BT, FP8SUMS, CFG, true>(g, s)
                    : launch_block_gemm_pipe<FA, FB, BT, FP8SUMS, CFG, false>(g, s);
}

// The kernel for a product.  us measured on an MI355X, N = 4096 and FP8 sums where not said otherwise, operands taking
// turns beyond what the last-level cache holds.
template <int FA, int FB, bool BT, bool FP8SUMS>
hipError_t launch_block_gemm_as(BlockGemmArgs g, hipStream_t s) {
    // All but the general kernel load straight to LDS: rows of whole aligned 16 bytes, offsets in 31 bits.
    if (g.M == 1) g.lda = (g.K + 15) / 16 * 16;  // a single row has no stride
    if (g.N == 1) g.ldb = (g.K + 15) / 16 * 16;
    const int64_t nk = (g.K + kBlk - 1) / kBlk, lim = (int64_t)1 << 31;
    const int64_t lim_code = lim / 256, lim_scale = (lim / 4 - 257) / nk;  // strides may be any 64-bit number: no products
    const bool aligned = g.lda % 16 == 0 && g.ldb % 16 == 0 && (uintptr_t)g.a % 16 == 0 && (uintptr_t)g.b % 16 == 0 &&
                         g.lda < lim_code && g.ldb < lim_code && g.ldsa <= lim_scale && g.ldsb <= lim_scale;
    const auto general = [&]() {
        g.tiles_m = (g.M + GB - 1) / GB;
        g.tiles_n = (g.N + GB - 1) / GB;
        hipLaunchKernelGGL((k_block_gemm<FA, FB, BT, FP8SUMS>), dim3((unsigned)(g.tiles_m * g.tiles_n)), dim3(GNT), 0, s, g);
        return hipGetLastError();
    };
    if (!aligned) return general();
    const auto tiles = [&](int64_t m, int64_t n) { return (g.M + m - 1) / m * ((g.N + n - 1) / n); };
    const int64_t wide = (int64_t)1 << 26;  // columns from which 16 of them per workgroup would be 2^31 threads
    if (g.M <= 8 && g.N < wide) return launch_block_gemm_few<FA, FB, BT, FP8SUMS, 1, 1, 2>(g, s);
    if (g.M <= 16 && g.N < wide) return launch_block_gemm_few<FA, FB, BT, FP8SUMS, 2, 1, 2>(g, s);
    if (g.M <= 32 && g.N < wide) return launch_block_gemm_few<FA, FB, BT, FP8SUMS, 4, 1, 3>(g, s);
    if (g.M <= 48 && g.N < wide) return launch_block_gemm_few<FA, FB, BT, FP8SUMS, 6, 1, 2>(g, s);
    // 64 rows: 32 columns per workgroup read A half as often, 16 make twice the workgroups, one per CU either way.  16
    // while that is one round: K = 14336, N = 4096 (256 workgroups of 16) 25.7 against 30; K = 4096, N = 6144 (384) 13.8
    // against 9.6, 8192 (512) 16.7 against 12, 28672 (1792) 56 against 44.
    if (g.M <= 64 && tiles(64, 16) <= 256) return launch_block_gemm_few<FA, FB, BT, FP8SUMS, 8, 1, 1>(g, s);
    // Up to two rounds of 64 x 32 tiles on the 256 CUs (the 128 x 128 tiles are then 64 at most): K = 14336, one
    // round (M = 128) 30 against 92, two (256) 49 against 90; K = 4096, one 9.2 against 19.6, two 16.6 against 20,
    // four (512) 30 against 20.5.  fp32 sums, K = 4096: one 10.6 against 31, two 19 against 31, four 34 against 32.
    if ((g.M <= 64 && g.N < wide) || tiles(64, 32) <= 512) return launch_block_gemm_few<FA, FB, BT, FP8SUMS, 8, 2, 1>(g, s);
    if (g.K < 16) return general();  // no whole chunk for a stage
    const int64_t r128 = (tiles(128, 128) + 255) / 256;
    if constexpr (FP8SUMS && BT) {
        // a round of 256 x 256 tiles takes 1.75 us per 128 K, one of 128 x 128 tiles 0.70
        const int64_t r256 = (tiles(256, 256) + 255) / 256;
        if (5 * r256 <= 2 * r128) return launch_block_gemm_k<FA, FB, BT, FP8SUMS, Cfg256x256>(g, s);
        // long rows, every CU busy: 1000 rows, operands from HBM, K = 28672 180 without and 155 with the prefetch;
        // 14336 91 and 82; 12288 81 and 76; 8192 43 and 45.  (Operands that the last-level cache holds: 14336 72
        // and 78.)
        if (g.K >= 12288 && tiles(128, 128) >= 256)
            return launch_block_gemm_k<FA, FB, BT, FP8SUMS, Cfg128x128Far>(g, s);
    } else {
        // (with fp32 sums or B's scales by column 256 x 256 tiles need more registers than there are)
        // a round of 256 x 128 tiles takes 2.0 us per 128 K (fp32 sums), one of 128 x 128 tiles 1.05; FP8 sums, B's
        // scales by column: 1.3 and 0.70 (6144 x 4096 x 8192 in 3 rounds 249, in 6 of 128 x 128 tiles 271; 1536 x
        // 4096 x 4096 in one 44, in two 50; 1024 x 4096 x 4096 in one of either 38 and 29)
        const int64_t r256 = (tiles(256, 128) + 255) / 256;
        if (2 * r256 <= r128) return launch_block_gemm_k<FA, FB, BT, FP8SUMS, Cfg256x128>(g, s);
    }
    return launch_block_gemm_k<FA, FB, BT, FP8SUMS, Cfg128x128>(g, s);
}

template <int FA, int FB>
hipError_t launch_block_gemm_fmt(const BlockGemmArgs &g, bool bt, bool fp8_sums, hipStream_t s) {
    if (bt) return fp8_sums ? launch_block_gemm_as<FA, FB, true, true>(g, s) : launch_block_gemm_as<FA, FB, true, false>(g, s);
    return fp8_sums ? launch_block_gemm_as<FA, FB, false, true>(g, s) : launch_block_gemm_as<FA, FB, false, false>(g, s);
}

}  // namespace
}  // namespace mx
