// mx_block_quant.hip -- block-128 FP8 quantizers for gfx950: bf16 to E4M3 or
// E5M2 codes with one fp32 scale for each block of 128 along the rows, along
// the columns (written transposed), or for each 128 x 128 tile; both forms from
// one read.
//
// A workgroup takes one 128 x 128 tile of x, so every block it meets lies
// inside it whole.  Thread (rg, cg) holds the 8 x 8 patch of rows 8 rg .. and
// columns 8 cg ..: a wave's load instruction reads 256 contiguous bytes of each
// of four rows; a row block's amax is a maximum over the 16 lanes of a DPP row;
// a column block's is one over the thread's 8 rows, the wave's 4 row groups and
// the 4 waves (LDS).  The row form is written from the registers, 128-byte runs;
// the transposed form goes through LDS, 8 codes of a column at a time, and
// leaves as 128-byte runs of its own rows.  Scales leave as runs too, since the
// reduction dimension's blocks are their outer dimension.
//
// Bound by memory: 2 bytes read and 1 byte (and 1/32) written per element and
// form.  Measured over inputs and outputs that take turns: 28672 x 4096 in tiles,
// both forms (470 MB) 92 us, 5.1 TB/s as a large copy (75 where the outputs go
// over the same memory call after call, which the last-level cache then holds);
// 8192 x 4096 by rows (102 MB) 21 us (18.6 over the same outputs); 1000 x 6144, both
// forms (25 MB, 384 workgroups) 10.4 us, of which launch, one read's latency, two
// barriers and the stores, one after the other, are the most.
#include "mx_block_util.h"

namespace mx {
namespace {

constexpr int kQT = 256;

template <int FR, int FT, bool ROW, bool TR, bool TILE, bool WHOLE, bool NT>
__global__ __launch_bounds__(kQT) void k_block_quantize(const uint16_t *__restrict__ x, int64_t rows, int64_t cols,
                                                        int64_t ldx, uint32_t tiles_c, FastDiv tc_div, BlockForm fr,
                                                        BlockForm ft) {
    __shared__ __attribute__((aligned(16))) uint8_t sT[TR ? kBlk * kBlk : 16];
    __shared__ __attribute__((aligned(16))) uint32_t sM[4][16][4];
    const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4, wave = tid >> 6;
    const uint32_t tr_i = tc_div.div(blockIdx.x), tc_i = blockIdx.x - tr_i * tiles_c;
    const int64_t r0 = (int64_t)tr_i * kBlk, c0 = (int64_t)tc_i * kBlk;
    const int nr = (int)min((int64_t)kBlk, rows - r0), nc = (int)min((int64_t)kBlk, cols - c0);
    const int nrt = nr - 8 * rg, nct = nc - 8 * cg;  // this thread's rows and columns inside the matrix (may be <= 0)

    uint32_t w[8][4];
    const uint16_t *const px = x + r0 * ldx + c0;  // scalar; a row of the tile is a 32-bit step from it
#pragma unroll
    for (int i = 0; i < 8; i++)  // a row past the matrix reads the tile's first one and counts as zeros
        load_vec<WHOLE, NT>(w[i], px + (i < nrt ? (int64_t)(8 * rg + i) * ldx : 0), 8 * cg, nc, i < nrt);

    float inv_t[TR ? 8 : 1];
    bool ok_t[TR ? 8 : 1];
    float inv_tile = 0.f, inv_tile_t = 0.f;
    bool ok_tile = true;
    if constexpr (TILE || TR) {
        uint32_t m[4] = {0, 0, 0, 0};  // largest magnitudes of the thread's columns, two per word
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int k = 0; k < 4; k++) m[k] = pk_max_u16(m[k], w[i][k] & 0x7FFF7FFFu);
#pragma unroll
        for (int k = 0; k < 4; k++) {
            m[k] = pk_max_u16(m[k], (uint32_t)__shfl_xor((int)m[k], 16));
            m[k] = pk_max_u16(m[k], (uint32_t)__shfl_xor((int)m[k], 32));
        }
        if ((tid & 48) == 0) *reinterpret_cast<uint4 *>(sM[wave][cg]) = make_uint4(m[0], m[1], m[2], m[3]);
        __syncthreads();
#pragma unroll
        for (int v = 0; v < 4; v++) {
            const uint4 t = *reinterpret_cast<const uint4 *>(sM[v][cg]);
            m[0] = pk_max_u16(m[0], t.x);
            m[1] = pk_max_u16(m[1], t.y);
            m[2] = pk_max_u16(m[2], t.z);
            m[3] = pk_max_u16(m[3], t.w);
        }
        if constexpr (TILE) {
            uint32_t a = row16_max_pk(pk_max_u16(pk_max_u16(m[0], m[1]), pk_max_u16(m[2], m[3])));
            a = umax(a & 0xFFFFu, a >> 16);
            float s, st;
            block_scale<FR>(a << 16, s, inv_tile, ok_tile);
            block_scale<FT>(a << 16, st, inv_tile_t, ok_tile);
            if (tid == 0) {
                if constexpr (ROW) fr.scales[(int64_t)tc_i * fr.ld_scales + tr_i] = s;
                if constexpr (TR) ft.scales[(int64_t)tr_i * ft.ld_scales + tc_i] = st;
            }
        } else {
            float s[8];
#pragma unroll
            for (int j = 0; j < 8; j++)
                block_scale<FT>((j & 1) ? (m[j >> 1] & 0xFFFF0000u) : (m[j >> 1] << 16), s[j], inv_t[j], ok_t[j]);
            if (rg == 0) {
                float *d = ft.scales + (int64_t)tr_i * ft.ld_scales + c0 + 8 * cg;
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (j < nct) d[j] = s[j];
            }
        }
    }

    if constexpr (ROW) {
        uint8_t *q = fr.codes + (r0 + 8 * rg) * fr.ld_codes + c0 + 8 * cg;
        float s[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float inv[2];
            bool ok[2];
            if constexpr (TILE) {
                inv[0] = inv[1] = inv_tile;
                ok[0] = ok[1] = ok_tile;
            } else {
                uint32_t ra = 0, rb = 0;  // rows i and i + 1, then one in each half
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    ra = pk_max_u16(ra, w[i][k] & 0x7FFF7FFFu);
                    rb = pk_max_u16(rb, w[i + 1][k] & 0x7FFF7FFFu);
                }
                const uint32_t m = row16_max_pk(pk_max_u16(__builtin_amdgcn_perm(rb, ra, 0x05040100u),
                                                           __builtin_amdgcn_perm(rb, ra, 0x07060302u)));
                block_scale<FR>(m << 16, s[i], inv[0], ok[0]);
                block_scale<FR>(m & 0xFFFF0000u, s[i + 1], inv[1], ok[1]);
            }
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const uint32_t(&v)[4] = w[i + e];
                const uint32_t lo = block_cvt4<FR>(bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1]), inv[e], ok[e]);
                const uint32_t hi = block_cvt4<FR>(bf16_lo(v[2]), bf16_hi(v[2]), bf16_lo(v[3]), bf16_hi(v[3]), inv[e], ok[e]);
                if (i + e < nrt && nct > 0) {
                    if (WHOLE) {
                        const uint32_t t[2] = {lo, hi};
                        __builtin_memcpy(q + (i + e) * fr.ld_codes, t, 8);
                    } else {
                        store8(q + (i + e) * fr.ld_codes, lo, hi, nct);
                    }
                }
            }
        }
        if constexpr (!TILE) {
            if (cg == 0) {
                float *d = fr.scales + (int64_t)tc_i * fr.ld_scales + r0 + 8 * rg;
#pragma unroll
                for (int i = 0; i < 8; i++)
                    if (i < nrt) d[i] = s[i];
            }
        }
    }

    if constexpr (TR) {
        // codes of column c, rows 8 rg .. +7, at 8-byte slot rg ^ (c >> 3) of LDS row c.  Odd
        // column groups take their columns in pairs swapped, so that the 16 groups of one
        // write spread over both halves of the 64 banks.
#pragma unroll
        for (int jj = 0; jj < 8; jj++) {
            uint32_t lo[2], hi[2];
            // both columns of the pair are converted once; the select is on the group's parity
            if (jj & 1) continue;
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int j = jj + e, k = j >> 1;
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; i++) y[i] = (j & 1) ? bf16_hi(w[i][k]) : bf16_lo(w[i][k]);
                const float inv = TILE ? inv_tile_t : inv_t[TILE ? 0 : j];
                const bool ok = TILE ? ok_tile : ok_t[TILE ? 0 : j];
                lo[e] = block_cvt4<FT>(y[0], y[1], y[2], y[3], inv, ok);
                hi[e] = block_cvt4<FT>(y[4], y[5], y[6], y[7], inv, ok);
            }
            const int odd = cg & 1;
            const int slot = ((rg ^ cg) & 15) << 3;
            const int ca = 8 * cg + jj + odd, cb = 8 * cg + jj + 1 - odd;
            *reinterpret_cast<uint2 *>(&sT[ca * kBlk + slot]) = odd ? make_uint2(lo[1], hi[1]) : make_uint2(lo[0], hi[0]);
            *reinterpret_cast<uint2 *>(&sT[cb * kBlk + slot]) = odd ? make_uint2(lo[0], hi[0]) : make_uint2(lo[1], hi[1]);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int t = k * kQT + tid, c = t >> 3, q = t & 7, g = c >> 3;
            if (c >= nc || 16 * q >= nr) continue;
            const uint4 v = *reinterpret_cast<const uint4 *>(&sT[c * kBlk + ((q ^ (g >> 1)) << 4)]);
            const uint4 u = (g & 1) ? make_uint4(v.z, v.w, v.x, v.y) : v;
            uint8_t *d = ft.codes + (c0 + c) * ft.ld_codes + r0 + 16 * q;
            if (16 * q + 16 <= nr) {
                __builtin_memcpy(d, &u, 16);
            } else {
                store8(d, u.x, u.y, min(8, nr - 16 * q));
                store8(d + 8, u.z, u.w, nr - 16 * q - 8);
            }
        }
    }
}

template <bool TILE>
hipError_t launch_forms(const uint16_t *x, int64_t rows, int64_t cols, int64_t ldx, const BlockForm &r,
                        const BlockForm &t, hipStream_t s) {
    const uint32_t tc = (uint32_t)((cols + kBlk - 1) / kBlk), trn = (uint32_t)((rows + kBlk - 1) / kBlk);
    const dim3 grid(tc * trn), block(kQT);
    const FastDiv d(tc);
    // Input larger than half of the 256 MB last-level cache is read past it: less of it would be found there
    // than it pushes out.  Through the cache and past it, with outputs over the same memory call after call:
    // 28672 x 4096 in tiles, both forms 91 and 75 us, 8192 x 4096 (67 MB, partly still cached), one form 18.6 and
    // 20.0; with outputs in turn 92 either way, and 21.3 and 20.0.
    const bool whole = cols % 8 == 0, nt = whole && rows * cols > (int64_t)1 << 26;
#define MX_Q(fr, ft, row, tr)                                                                                             \
    do {                                                                                                                  \
        if (nt) hipLaunchKernelGGL((k_block_quantize<fr, ft, row, tr, TILE, true, true>), grid, block, 0, s, x, rows,     \
                                   cols, ldx, tc, d, r, t);                                                               \
        else if (whole) hipLaunchKernelGGL((k_block_quantize<fr, ft, row, tr, TILE, true, false>), grid, block, 0, s, x,  \
                                           rows, cols, ldx, tc, d, r, t);                                                 \
        else hipLaunchKernelGGL((k_block_quantize<fr, ft, row, tr, TILE, false, false>), grid, block, 0, s, x, rows,      \
                                cols, ldx, tc, d, r, t);                                                                  \
    } while (0)
    if (r.codes && t.codes) {
        switch (r.fmt * 2 + t.fmt) {
        case 0: MX_Q(0, 0, true, true); break;
        case 1: MX_Q(0, 1, true, true); break;
        case 2: MX_Q(1, 0, true, true); break;
        default: MX_Q(1, 1, true, true); break;
        }
    } else if (r.codes) {
        if (r.fmt == E4M3) MX_Q(0, 0, true, false);
        else MX_Q(1, 1, true, false);
    } else {
        if (t.fmt == E4M3) MX_Q(0, 0, false, true);
        else MX_Q(1, 1, false, true);
    }
#undef MX_Q
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_quantize(const uint16_t *x, int64_t rows, int64_t cols, int64_t ldx, bool tile,
                                 const BlockForm &row, const BlockForm &tr, hipStream_t stream) {
    return tile ? launch_forms<true>(x, rows, cols, ldx, row, tr, stream)
                : launch_forms<false>(x, rows, cols, ldx, row, tr, stream);
}

}  // namespace mx
