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
template <bool WHOLE>
__device__ __forceinline__ void load_vec(uint32_t (&w)[4], const uint16_t *p, int c, int cols, bool live) {
    if constexpr (WHOLE) {
        __builtin_memcpy(w, reinterpret_cast<const uint8_t *>(p) + 2u * (uint32_t)min(c, cols - 8), 16);
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

// max over the 16 lanes of a DPP row, in every one of them: neighbours, pairs, halves mirrored, whole row mirrored
__device__ __forceinline__ uint32_t row16_max_pk(uint32_t v) {
    v = pk_max_u16(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));
    v = pk_max_u16(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));
    v = pk_max_u16(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));
    v = pk_max_u16(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));
    return v;
}
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    v = quad_max(v);
    v = umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));
    v = umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));
    return v;
}

// scale and inverse of a block from its amax bits (fp32 magnitude).  A block
// with an Inf or NaN has scale NaN; ok = false then zeroes its codes.
template <int F>
__device__ __forceinline__ void block_scale(uint32_t amax_bits, float &scale, float &inv, bool &ok) {
    ok = amax_bits < 0x7F800000u;
    const float amax = __builtin_fmaxf(__uint_as_float(ok ? amax_bits : 0u), kAmaxFloor);
    scale = ok ? amax / block_fmax<F>() : __uint_as_float(0x7FC00000u);
    inv = block_fmax<F>() / amax;
}

// four codes of v * inv, clamped to the format's largest value
template <int F>
__device__ __forceinline__ uint32_t block_cvt4(float a, float b, float c, float d, float inv, bool ok) {
    const uint32_t q = cvt4_fp8<F>(a * inv, b * inv, c * inv, d * inv, 1.0f, block_fmax<F>());
    return ok ? q : 0u;
}

}  // namespace
}  // namespace mx
