// mx_block_util.h -- device helpers shared by the block-128 quantizer and the
// norm: loads and stores of partial vectors, 16-lane maxima, scales and casts.
#pragma once
#include "mx_block_internal.h"
#include "mx_quant_kernels.h"

namespace mx {
namespace {

// The target allows unaligned global accesses, so a whole vector is one
// instruction at any address; only a vector that the row's end cuts is taken
// element by element (past the end nothing is touched).

// 8 bf16 from p, n of them valid (the rest 0), two per word
__device__ __forceinline__ void load8_bf16(uint32_t (&w)[4], const uint16_t *p, int n) {
    if (n >= 8) {
        __builtin_memcpy(w, p, 16);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t lo = 2 * i < n ? p[2 * i] : 0u, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0u;
            w[i] = lo | (hi << 16);
        }
    }
}

// Vector c .. c + 7 of a row of cols elements at p, zeros past its end and for a row that is not live
// (p is then any readable row).  A scalar row address and an unsigned 32-bit lane offset make one
// load without 64-bit vector arithmetic.  WHOLE: cols is a multiple of 8, so a vector lies in the row or past it;
// the load is unconditional (from the row's last vector where it lies past it) and the zeros a select:
// a branch per load would keep the loads of a row from going out together.
// NT: read past the caches.
template <bool WHOLE, bool NT = false>
__device__ __forceinline__ void load_vec(uint32_t (&w)[4], const uint16_t *p, int c, int cols, bool live) {
    if constexpr (WHOLE) {
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
        const u32x4 *q = reinterpret_cast<const u32x4 *>(reinterpret_cast<const uint8_t *>(p) + 2u * (uint32_t)min(c, cols - 8));
        const u32x4 t = NT ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
        for (int k = 0; k < 4; k++) w[k] = t[k];
        const bool in = live && c < cols;
#pragma unroll
        for (int k = 0; k < 4; k++) w[k] = in ? w[k] : 0u;
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++) w[k] = 0u;
        if (live && c < cols) load8_bf16(w, p + (uint32_t)c, cols - c);
    }
}

// the first n of 8 bytes
__device__ __forceinline__ void store8(uint8_t *p, uint32_t lo, uint32_t hi, int n) {
    if (n >= 8) {
        const uint32_t v[2] = {lo, hi};
        __builtin_memcpy(p, v, 8);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n) p[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
}

// v from another lane of its row of 16.  Every lane has a source in the patterns below; said so (the last
// argument), the compiler folds the move into the operation that takes it.
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
// max over the 16 lanes of a DPP row, in every one of them: neighbours, pairs, halves mirrored, whole row mirrored
__device__ __forceinline__ uint32_t row16_max_pk(uint32_t v) {
    v = pk_max_u16(v, dpp<kDppXor1>(v));
    v = pk_max_u16(v, dpp<kDppXor2>(v));
    v = pk_max_u16(v, dpp<kDppHalfMirror>(v));
    return pk_max_u16(v, dpp<kDppMirror>(v));
}
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    v = umax(v, dpp<kDppXor1>(v));
    v = umax(v, dpp<kDppXor2>(v));
    v = umax(v, dpp<kDppHalfMirror>(v));
    return umax(v, dpp<kDppMirror>(v));
}

// scale and inverse of a block from its amax bits (fp32 magnitude).  A block
// with an Inf or NaN has scale NaN; ok = false then zeroes its codes.
//
// Both quotients are correctly rounded: an approximation, then one correction by its exact remainder (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990), 10 operations for the two
// where the compiler's division takes about 12 for each.  amax / 2^12 keeps the reciprocal and every
// intermediate in fp32's normal range.  Compared with `/` on the device: equal for every fp32 from 2^-100 up.
template <int F>
__device__ __forceinline__ void block_scale(uint32_t amax_bits, float &scale, float &inv, bool &ok) {
    constexpr float fmax = block_fmax<F>(), rf = 1.0f / fmax;
    ok = amax_bits < 0x7F800000u;
    const float amax = __builtin_fmaxf(__uint_as_float(ok ? amax_bits : 0u), kAmaxFloor);
    const float s0 = amax * rf;
    const float s1 = __builtin_fmaf(__builtin_fmaf(-s0, fmax, amax), rf, s0);
    scale = ok ? s1 : __uint_as_float(0x7FC00000u);
    const float a = amax * 0x1p-12f;
    const float y0 = __builtin_amdgcn_rcpf(a);
    const float y1 = __builtin_fmaf(__builtin_fmaf(-a, y0, 1.0f), y0, y0);
    const float q0 = fmax * y1;
    inv = __builtin_fmaf(__builtin_fmaf(-a, q0, fmax), y1, q0) * 0x1p-12f;
}

// Four codes of v * inv.  No clamp: where ok, |v| <= amax and inv <= (1 + 2^-23) fmax / amax, so that |v * inv|
// exceeds the largest code by 2^-22 of it at most and rounds to it.
template <int F>
__device__ __forceinline__ uint32_t block_cvt4(float a, float b, float c, float d, float inv, bool ok) {
    v2s w = {0, 0};
    if constexpr (F == E4M3) {
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a * inv, b * inv, 1.0f, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c * inv, d * inv, 1.0f, true);
    } else {
        w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w, a * inv, b * inv, 1.0f, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w, c * inv, d * inv, 1.0f, true);
    }
    return ok ? __builtin_bit_cast(uint32_t, w) : 0u;
}

}  // namespace
}  // namespace mx
