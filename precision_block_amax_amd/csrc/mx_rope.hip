// mx_rope.hip -- rotary positions of queries and keys for gfx950, alone or after
// the RMS norm of each head in one pass, and the backward pass of both.
//
// Rotation at position p: pair i (a, b) of a head becomes (a c - b s, b c + a s),
// c, s = scale * (cos, sin)(p * freq_i).  Its transpose, the backward pass, is the
// rotation by the opposite angle.  The angle is taken in fp64 as turns, p * freq_i /
// 2 pi less the nearest whole number: what is left is exact to p * 2^-53 turns,
// then rounded to fp32, 2^-25 of a turn, 2^-23 of its radius (fp32 products of far
// positions, 2^17 and more, would be off by 2^-8 and more).  One lane makes one
// angle; they go through LDS to the lanes that need them, for all heads of a wave.
//
// Norm: xh = x * rstd, rstd = 1 / sqrt(mean(x^2) + eps) over the head, y = rope(xh * w).
// Backward, with u = inverse rotation of dy, g = u * w:
//   dx = rstd * (g - xh * mean(g * xh)),  dw = sum over tokens and heads of u * xh
// rstd is made again from x, which is read anyway.  The sums of dw stay in registers
// for all heads that a wave meets, then go through the workspace to a second kernel;
// every sum is in a fixed order, so the same inputs give the same bits.
//
// A wave takes heads of one token, 64 / L at a time: a head is 16 elements of
// each of L lanes, two vectors of eight.  In the half layout these are the two
// halves of eight pairs, so pairs never cross lanes and a head's sums are a DPP tree
// over L lanes.  Everything is fp32 until the one rounding to bf16.
//
// Bound by memory: 2 bytes read and 2 written per element, backward 4 and 2.  Measured
// with inputs in turn, heads of 128: rotation of 8192 tokens x 72 heads (302 MB) 50 us,
// 6.0 TB/s; norm and rotation of 8192 x 40 (168 MB) 27 to 29 us, 6.0 TB/s, backward (252 MB)
// 52 to 54 us, 4.8 TB/s, and 4 to 5 for the weights' sums; of 32768 x 40 114 us and 197 in all.  A copy
// reaches 5.2 from HBM; part of these inputs is still in the last-level cache.
// One token: 2.5 us, launch and latency.
#include <type_traits>

#include "mx_block_util.h"
#include "mx_rope_internal.h"

namespace mx {
namespace {

constexpr int kHW = 4;  // waves of a workgroup
constexpr int kMaxPairs = kHeadMaxDim / 2;

// sum over groups of L neighbouring lanes, in every lane of the group
template <int L>
__device__ __forceinline__ float group_sum(float v) {
    const auto add = [&](auto ctrl) { v += __uint_as_float(dpp<decltype(ctrl)::value>(__float_as_uint(v))); };
    if constexpr (L >= 2) add(std::integral_constant<int, kDppXor1>{});
    if constexpr (L >= 4) add(std::integral_constant<int, kDppXor2>{});
    if constexpr (L >= 8) add(std::integral_constant<int, kDppHalfMirror>{});
    if constexpr (L >= 16) add(std::integral_constant<int, kDppMirror>{});
    if constexpr (L >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if constexpr (L >= 64) {
        const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(q[0]) + __uint_as_float(q[1]);
    }
    return v;
}

// How a head lies in L lanes.  A lane has NS = 2 H slots, slot i and i + H (half layout) or 2 i and 2 i + 1
// (interleaved) a pair.  V > 0: slots are two vectors of V elements, from o0 and o1 on, all of its pairs rotated or
// none.  V = 0, any dim and rot: every pair is (i, i + H); the first four of a lane are pairs lane + 64 i of the
// rotation, the others elements behind it.
template <int V, int L, bool INTER>
struct Map {
    static constexpr int H = V ? V : 8, NS = 2 * H;
    static constexpr bool kPairwise = INTER && V == 1;  // a vector of one element holds no pair
    int o0, o1, l;
    bool act, rot;  // (V > 0) the lane has elements; they are rotated
    int dim, pairs, nrot;

    __device__ __forceinline__ Map(int lane, int dim_, int rot_) : dim(dim_), pairs(rot_ / 2), nrot(rot_) {
        l = lane % L;
        if constexpr (V > 0) {
            act = 2 * V * l < dim;
            rot = 2 * V * l < nrot;
            // neighbouring lanes' vectors lie side by side, those of the rotated part and those of the rest, in either
            // layout (with a lane's two vectors side by side, two loads read every line: interleaved, 8192 tokens
            // of 40 heads of 128, backward 64 us, forward 32)
            const int k = rot ? l : l - nrot / (2 * V), base = rot ? 0 : nrot, half = (rot ? nrot : dim - nrot) / 2;
            o0 = kPairwise && rot ? 2 * l : base + V * k;
            o1 = kPairwise && rot ? 2 * l + 1 : base + half + V * k;
        } else {
            act = rot = true;
            o0 = o1 = 0;
        }
    }
    // element of a slot, -1: none
    __device__ __forceinline__ int elem(int s) const {
        if constexpr (V > 0) return !act ? -1 : s < V ? o0 + s : o1 + s - V;
        const int i = s & 7, second = s >> 3;
        if (i < 4) {
            const int j = l + 64 * i;
            return j < pairs ? (INTER ? 2 * j + second : j + second * pairs) : -1;
        }
        const int e = nrot + l + 64 * (i - 4 + 4 * second);
        return e < dim ? e : -1;
    }

    // a lane's bf16 elements as they are in memory, zeros where there are none: two per word, or one (V = 0, 1)
    static constexpr int RAW = V > 1 ? V : NS;
    // NT: past the caches
    typedef uint32_t Vec __attribute__((ext_vector_type(V > 1 ? V / 2 : 1), aligned(2)));
    template <bool NT>
    __device__ __forceinline__ void fetch(uint32_t (&w)[RAW], const uint16_t *p, bool live) const {
        if constexpr (V > 1) {
            Vec a = {}, b = {};
            if (live && act) {
                const Vec *const pa = reinterpret_cast<const Vec *>(p + o0), *const pb = reinterpret_cast<const Vec *>(p + o1);
                a = NT ? __builtin_nontemporal_load(pa) : *pa;
                b = NT ? __builtin_nontemporal_load(pb) : *pb;
            }
#pragma unroll
            for (int i = 0; i < V / 2; i++) {
                w[i] = a[i];
                w[V / 2 + i] = b[i];
            }
        } else {
#pragma unroll
            for (int s = 0; s < NS; s++) {
                const int e = elem(s);
                w[s] = live && e >= 0 ? (uint32_t)p[e] : 0u;
            }
        }
    }
    __device__ __forceinline__ void unpack(float (&v)[NS], const uint32_t (&w)[RAW]) const {
        if constexpr (V > 1) {
#pragma unroll
            for (int i = 0; i < V; i++) {
                v[2 * i] = bf16_lo(w[i]);
                v[2 * i + 1] = bf16_hi(w[i]);
            }
        } else {
#pragma unroll
            for (int s = 0; s < NS; s++) v[s] = bf16_lo(w[s]);
        }
    }
    __device__ __forceinline__ void load(float (&v)[NS], const uint16_t *p, bool live) const {
        uint32_t w[RAW];
        fetch<false>(w, p, live);
        unpack(v, w);
    }
    template <bool NT>
    __device__ __forceinline__ void store(uint16_t *p, const float (&v)[NS], bool live) const {
        if constexpr (V > 1) {
            Vec a, b;
#pragma unroll
            for (int i = 0; i < V / 2; i++) {
                a[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{v[2 * i], v[2 * i + 1]}, v2bf));
                b[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{v[V + 2 * i], v[V + 2 * i + 1]}, v2bf));
            }
            Vec *const pa = reinterpret_cast<Vec *>(p + o0), *const pb = reinterpret_cast<Vec *>(p + o1);
            if (live && act) {
                if constexpr (NT) {
                    __builtin_nontemporal_store(a, pa);
                    __builtin_nontemporal_store(b, pb);
                } else {
                    *pa = a;
                    *pb = b;
                }
            }
        } else {
#pragma unroll
            for (int s = 0; s < NS; s++) {
                const int e = elem(s);
                const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{v[s], 0.f}, v2bf));
                if (live && e >= 0) p[e] = (uint16_t)w;
            }
        }
    }
    // a weight of the head's elements as fp32, 1 where there is none
    __device__ __forceinline__ void load_weight(float (&v)[NS], const void *p, bool bf16) const {
#pragma unroll
        for (int s = 0; s < NS; s++) v[s] = 1.f;
        if (!p) return;
        if (bf16) {
            load(v, reinterpret_cast<const uint16_t *>(p), true);
            return;
        }
        const float *const q = reinterpret_cast<const float *>(p);
        if constexpr (V > 1) {
            if (act) {
                __builtin_memcpy(&v[0], q + o0, 4 * V);
                __builtin_memcpy(&v[V], q + o1, 4 * V);
            }
        } else {
#pragma unroll
            for (int s = 0; s < NS; s++) {
                const int e = elem(s);
                v[s] = e >= 0 ? q[e] : 0.f;
            }
        }
    }

    // cosines and sines of the lane's pairs
    __device__ __forceinline__ void angles(float2 (&cs)[H], const float2 *all) const {
#pragma unroll
        for (int i = 0; i < H; i++) {
            // the lane's slots are elements V l .. and pairs + V l ..: of the half layout the pairs V l .., of the
            // interleaved one V l / 2 .. and as many from (pairs + V l) / 2 on
            if constexpr (V > 1 && INTER) cs[i] = all[!rot ? 0 : i < V / 2 ? V / 2 * l + i : pairs / 2 + V / 2 * l + i - V / 2];
            else if constexpr (V > 0) cs[i] = all[rot ? V * l + i : 0];
            else cs[i] = all[i < 4 && l + 64 * i < pairs ? l + 64 * i : 0];
        }
    }
    // v: rotated in place; sign -1: the other way round
    __device__ __forceinline__ void rotate(float (&v)[NS], const float2 (&cs)[H], float sign) const {
        const auto turn = [&](float &a, float &b, float2 t) {
            const float s = sign * t.y, u = __builtin_fmaf(a, t.x, -(b * s)), w = __builtin_fmaf(b, t.x, a * s);
            a = u;
            b = w;
        };
        if constexpr (V > 0) {
            if (rot) {
#pragma unroll
                for (int i = 0; i < V; i++) turn(v[INTER ? 2 * i : i], v[INTER ? 2 * i + 1 : i + V], cs[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (l + 64 * i < pairs) turn(v[i], v[i + 8], cs[i]);
        }
    }

    typedef float f2 __attribute__((ext_vector_type(2)));
};

// scale * (cos, sin) of every pair's angle at one position, into the wave's part of LDS
__device__ __forceinline__ void make_angles(float2 *cs, const RopeArgs &a, int64_t token, int lane) {
    if (a.rot == 0) return;  // there may be no positions
    const double pos = a.pos64 ? (double)reinterpret_cast<const int64_t *>(a.pos)[token]
                               : (double)reinterpret_cast<const int32_t *>(a.pos)[token];
    __builtin_amdgcn_wave_barrier();  // the angles of the token before have been read
    for (int i = lane; i < a.rot / 2; i += 64) {
        const double t = pos * a.freqs[i] * 0.15915494309189533577;  // 1 / (2 pi)
        float s, c;
        sincospif(2.0f * (float)(t - __builtin_rint(t)), &s, &c);
        cs[i] = make_float2(c * a.scale, s * a.scale);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A power of two that brings a head's squares back into fp32 where m, their mean plus eps, has left it (elements of 2^59
// and more) or lies where their small ones have (below 2^-100): for any finite bf16 elements the sum of the scaled
// squares is within 2^-66 .. 2^125, or zero.  1 for all others, whose bits it leaves alone.
__device__ __forceinline__ float head_factor(float m) {
    return m >= 0x1p-100f && m < INFINITY ? 1.f : m < 1.f ? 0x1p100f : 0x1p-70f;
}

// Forward.  A token's heads are passes of 64 / L, queries first, a wave for each: its own angles cost a wave less than
// waiting does for its next heads.  8192 tokens of 72 heads of 128, rotation: a wave for nine passes 65 us, for three
// 59.5, for two 57, for one 53 (5.7 TB/s); 40 heads, norm and rotation 28 for five, 27 for one.
// Lanes of fewer than 16 elements have as many passes more (8192 tokens of 40 heads of 128, 20 rotated: 139 us an element at a time, 27 so).
template <int V>
constexpr int kPasses = V == 0 ? 1 : 8 / V;
template <bool NORM, int V, int L, bool INTER, bool NT>
__global__ __launch_bounds__(64 * kHW) void k_heads(RopeArgs a, FastDiv parts, int passes) {
    typedef Map<V, L, INTER> M;
    constexpr int G = 64 / L;
    __shared__ float2 sCS[kHW][kMaxPairs];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t item = blockIdx.x * kHW + wave, tok = parts.div(item);
    if (tok >= a.tokens) return;  // a whole wave; no barriers of the workgroup below
    const int p0 = (int)(item - tok * parts.d) * kPasses<V>, pq = (a.s[0].heads + G - 1) / G;
    const M m(lane, a.dim, a.rot);
    make_angles(sCS[wave], a, tok, lane);
    float2 cs[M::H];
    m.angles(cs, sCS[wave]);
#pragma unroll
    for (int i = 0; i < kPasses<V>; i++) {
        const int p = p0 + i;
        if (p >= passes) break;
        const HeadSet &h = a.s[p >= pq];
        const int head = (p >= pq ? p - pq : p) * G + lane / L;
        const bool live = head < h.heads;
        float v[M::NS];
        m.load(v, h.x + tok * h.xt + head * h.xh, live);
        if constexpr (NORM) {
            float w[M::NS], sq = 0.f;
            m.load_weight(w, h.weight, a.param_bf16);
#pragma unroll
            for (int s = 0; s < M::NS; s++) sq = __builtin_fmaf(v[s], v[s], sq);
            const float rn = 1.0f / (float)a.dim;
            float m2 = __builtin_fmaf(group_sum<L>(sq), rn, a.eps);
            const float f = head_factor(m2);
            if (__any(f != 1.f)) {  // hardly ever; the whole wave, as group_sum moves across lanes
                sq = 0.f;
#pragma unroll
                for (int s = 0; s < M::NS; s++) {
                    v[s] *= f;
                    sq = __builtin_fmaf(v[s], v[s], sq);
                }
                m2 = __builtin_fmaf(group_sum<L>(sq), rn, a.eps * f * f);
            }
            const float rstd = rsqrt1(m2);
#pragma unroll
            for (int s = 0; s < M::NS; s++) v[s] = v[s] * rstd * w[s];
        }
        m.rotate(v, cs, !NORM && a.inverse ? -1.f : 1.f);
        m.template store<NT>(h.out + tok * h.ot + head * h.oh, v, live);
    }
}

// Backward of the norm and the rotation.  The first gq workgroups take the queries, the others the keys (a wave then
// has one weight and one sum of its gradient).  Waves take every so many-th token, so that what all of them read at a
// time lies together, and fetch the next pass's x and dy while they work on one.  8192 tokens of 40 heads of 128: 52 us; with
// a range of passes for each wave 66, with every so many-th pass instead of token 58 (32768
// tokens, interleaved: 226 and 263).
template <int V, int L, bool INTER, bool NT>
__global__ __launch_bounds__(64 * kHW, V ? 4 : 1) void k_heads_bwd(RopeArgs a, int gq) {
    typedef Map<V, L, INTER> M;
    constexpr int G = 64 / L;
    __shared__ union {
        float2 cs[kHW][kMaxPairs];
        float sum[kHW][kHeadMaxDim];
    } sh;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), sub = lane / L;
    const bool keys = (int)blockIdx.x >= gq;
    const HeadSet &h = a.s[keys];
    const int64_t step = (int64_t)(keys ? gridDim.x - gq : gq) * kHW;
    int64_t tok = (int64_t)(blockIdx.x - (keys ? gq : 0)) * kHW + wave;
    const M m(lane, a.dim, a.rot);
    const float rn = 1.0f / (float)a.dim;
    float acc[M::NS], w[M::NS];
    m.load_weight(w, h.weight, a.param_bf16);
#pragma unroll
    for (int s = 0; s < M::NS; s++) acc[s] = 0.f;
    uint32_t rx[M::RAW], rd[M::RAW];
    const auto fetch = [&](int64_t t, int p) {
        const int head = p + sub;
        const bool live = t < a.tokens && head < h.heads;
        m.template fetch<NT>(rx, h.x + t * h.xt + head * h.xh, live);
        m.template fetch<NT>(rd, h.dy + t * h.dt + head * h.dh, live);
    };
    fetch(tok, 0);
    for (; tok < a.tokens; tok += step) {
        make_angles(sh.cs[wave], a, tok, lane);
        uint16_t *const po = h.out + tok * h.ot;
        for (int p = 0; p < h.heads; p += G) {
            const int head = p + sub;
            const bool live = head < h.heads;
            float v[M::NS], u[M::NS];
            m.unpack(v, rx);
            m.unpack(u, rd);
            const bool more = p + G < h.heads;
            fetch(more ? tok : tok + step, more ? p + G : 0);
            {
                float2 cs[M::H];
                m.angles(cs, sh.cs[wave]);
                m.rotate(u, cs, -1.f);
            }
            float sq = 0.f, sg = 0.f;
#pragma unroll
            for (int s = 0; s < M::NS; s++) {
                sq = __builtin_fmaf(v[s], v[s], sq);
                sg = __builtin_fmaf(u[s] * w[s], v[s], sg);
            }
            sq = group_sum<L>(sq);
            sg = group_sum<L>(sg);
            float m2 = __builtin_fmaf(sq, rn, a.eps);
            const float f = live ? head_factor(m2) : 1.f;
            const bool scaled = __any(f != 1.f);
            if (scaled) {  // hardly ever
                sq = sg = 0.f;
#pragma unroll
                for (int s = 0; s < M::NS; s++) {
                    v[s] *= f;
                    sq = __builtin_fmaf(v[s], v[s], sq);
                    sg = __builtin_fmaf(u[s] * w[s], v[s], sg);
                }
                sg = group_sum<L>(sg);
                m2 = __builtin_fmaf(group_sum<L>(sq), rn, a.eps * f * f);
            }
            const float rstd = live ? rsqrt1(m2) : 0.f;  // of x * f
            const float mean = sg * rstd * rn;           // of g * xh
#pragma unroll
            for (int s = 0; s < M::NS; s++) {
                const float xh = v[s] * rstd;
                acc[s] = __builtin_fmaf(u[s], xh, acc[s]);
                v[s] = __builtin_fmaf(-xh, mean, u[s] * w[s]) * rstd;
            }
            if (scaled) {
#pragma unroll
                for (int s = 0; s < M::NS; s++) v[s] *= f;
            }
            m.template store<NT>(po + head * h.oh, v, live);
        }
    }
    if (!a.s[0].dw && !a.s[1].dw) return;
    __syncthreads();  // the angles are done with
#pragma unroll
    for (int s = 0; s < M::NS; s++) {
        float v = acc[s];
#pragma unroll
        for (int o = L; o < 64; o *= 2) v += __shfl_xor(v, o);
        const int e = m.elem(s);
        if (sub == 0 && e >= 0) sh.sum[wave][e] = v;
    }
    __syncthreads();
    float *const d = a.ws + (int64_t)blockIdx.x * a.dim;
    for (int i = threadIdx.x; i < a.dim; i += 64 * kHW) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kHW; w++) v += sh.sum[w][i];
        d[i] = v;
    }
}

// The workgroups' sums: 16 elements of one weight per workgroup, 64 groups of lanes taking every 64th row of the
// workspace, eight of them under way at a time.
constexpr int kSC = 16, kSR = 64, kSL = 8;
__global__ __launch_bounds__(kSC * kSR) void k_heads_dw(const float *ws, int gq, int gk, int dim, float *dwq, float *dwk) {
    __shared__ float s[kSR][kSC + 1];
    const int col = threadIdx.x % kSC, row = threadIdx.x / kSC, i = blockIdx.x * kSC + col;
    float *const out = blockIdx.y ? dwk : dwq;
    if (!out) return;  // the whole workgroup
    const int n = blockIdx.y ? gk : gq;
    const float *const p = ws + (blockIdx.y ? (int64_t)gq * dim : 0) + i;
    float v = 0.f;
    if (i < dim)
        for (int c = row; c < n; c += kSR * kSL) {
            float t[kSL];
#pragma unroll
            for (int k = 0; k < kSL; k++) t[k] = p[(int64_t)min(c + k * kSR, n - 1) * dim];
#pragma unroll
            for (int k = 0; k < kSL; k++) v += c + k * kSR < n ? t[k] : 0.f;
        }
    s[row][col] = v;
    __syncthreads();
    for (int half = kSR / 2; half > 0; half /= 2) {
        if (row < half) s[row][col] += s[row + half][col];
        __syncthreads();
    }
    if (row == 0 && i < dim) out[i] = s[0][col];
}

// Workgroups of the backward pass for queries and keys: 1024 in all, four per CU, shared by their passes, as far as there
// are tokens for their waves (6 + 1 heads, 8192 tokens: by heads 32 us, by passes 17).
constexpr int kBwdGroups = 1024;
void bwd_groups(int64_t tokens, int64_t pq, int64_t pk, int &gq, int &gk) {
    const int64_t most = (tokens + kHW - 1) / kHW, q = (kBwdGroups * pq + (pq + pk) / 2) / (pq + pk);
    const auto cut = [&](int64_t n, int64_t passes) { return (int)(passes > 0 ? n < 1 ? 1 : n < most ? n : most : 0); };
    gq = cut(q, pq);
    gk = cut(kBwdGroups - q, pk);
}

hipError_t launch_dw(const RopeArgs &a, int gq, int gk, hipStream_t s) {
    hipLaunchKernelGGL(k_heads_dw, dim3((unsigned)((a.dim + kSC - 1) / kSC), 2), dim3(kSC * kSR), 0, s, (const float *)a.ws, gq,
                       gk, a.dim, a.s[0].dw, a.s[1].dw);
    return hipGetLastError();
}

template <int V, int L, bool INTER, bool NT>
hipError_t launch_nt(const RopeArgs &all, int op, hipStream_t s) {
    constexpr int G = 64 / L;
    const int64_t pq = ((int64_t)all.s[0].heads + G - 1) / G, pk = ((int64_t)all.s[1].heads + G - 1) / G, passes = pq + pk;
    if (op == NORM_ROPE_BWD) {
        int gq, gk;
        bwd_groups(all.tokens, pq, pk, gq, gk);
        hipLaunchKernelGGL((k_heads_bwd<V, L, INTER, NT>), dim3((unsigned)(gq + gk)), dim3(64 * kHW), 0, s, all, gq);
        const hipError_t e = hipGetLastError();
        return e != hipSuccess || (!all.s[0].dw && !all.s[1].dw) ? e : launch_dw(all, gq, gk, s);
    }
    const int64_t parts = (passes + kPasses<V> - 1) / kPasses<V>;
    const int64_t most = ((int64_t)1 << 25) / parts;  // tokens per launch: waves and threads in 32 bits
    for (int64_t t = 0; t < all.tokens; t += most) {
        RopeArgs a = all;
        a.tokens = all.tokens - t < most ? all.tokens - t : most;
        a.pos = (const uint8_t *)a.pos + t * (a.pos64 ? 8 : 4);
        for (HeadSet &h : a.s) {
            h.x += t * h.xt;
            h.out += t * h.ot;
        }
        const dim3 grid((unsigned)((a.tokens * parts + kHW - 1) / kHW));
        if (op == ROPE) hipLaunchKernelGGL((k_heads<false, V, L, INTER, NT>), grid, dim3(64 * kHW), 0, s, a, FastDiv((uint32_t)parts), (int)passes);
        else hipLaunchKernelGGL((k_heads<true, V, L, INTER, NT>), grid, dim3(64 * kHW), 0, s, a, FastDiv((uint32_t)parts), (int)passes);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int V, int L, bool INTER>
hipError_t launch_as(const RopeArgs &a, int op, hipStream_t s) {
    // Outputs of more than 64 MB are written past the caches, and the backward pass's inputs read past them: what is
    // behind these tensors stays in the 256 MB last-level cache.  8192 tokens of 40 heads of 128 (84 MB), inputs in
    // turn: norm and rotation 35 and 28 us, backward 58 and 52 (outputs alone 56); 72 heads, rotation 67 and 65, and
    // with loads past the caches 68.
    const int64_t n = a.tokens * ((int64_t)a.s[0].heads + a.s[1].heads) * a.dim;
    if constexpr (V > 0)
        if (n > (int64_t)1 << 25) return launch_nt<V, L, INTER, true>(a, op, s);
    return launch_nt<V, L, INTER, false>(a, op, s);
}

template <bool INTER>
hipError_t launch_layout(const RopeArgs &a, int op, hipStream_t s) {
    if (a.dim % 16 == 0 && a.rot % 16 == 0) {
        if (a.dim <= 64) return launch_as<8, 4, INTER>(a, op, s);
        if (a.dim <= 128) return launch_as<8, 8, INTER>(a, op, s);
        if (a.dim <= 256) return launch_as<8, 16, INTER>(a, op, s);
        return launch_as<8, 32, INTER>(a, op, s);
    }
    if (a.dim % 8 == 0 && a.rot % 8 == 0 && a.dim <= 128) return launch_as<4, 16, INTER>(a, op, s);
    if (a.dim % 4 == 0 && a.rot % 4 == 0) {
        if (a.dim <= 64) return launch_as<2, 16, INTER>(a, op, s);
        if (a.dim <= 128) return launch_as<2, 32, INTER>(a, op, s);
        if (a.dim <= 256) return launch_as<2, 64, INTER>(a, op, s);
    }
    if (a.dim % 2 == 0 && a.dim <= 128) return launch_as<1, 64, INTER>(a, op, s);
    return launch_as<0, 64, INTER>(a, op, s);
}

}  // namespace

int64_t heads_workspace(int64_t tokens, int64_t heads_q, int64_t heads_k, int64_t dim) {
    // a row for each workgroup: kBwdGroups, one more where a set's share rounds to none
    const int64_t most = 2 * ((tokens + kHW - 1) / kHW);
    return heads_q + heads_k > 0 ? (most < kBwdGroups + 1 ? most : kBwdGroups + 1) * dim : 0;
}

hipError_t launch_heads(const RopeArgs &a, int op, hipStream_t s) {
    if (a.tokens > 0 && a.s[0].heads + (int64_t)a.s[1].heads > 0)
        return a.interleaved ? launch_layout<true>(a, op, s) : launch_layout<false>(a, op, s);
    return op == NORM_ROPE_BWD && (a.s[0].dw || a.s[1].dw) ? launch_dw(a, 0, 0, s) : hipSuccess;
}

}  // namespace mx
