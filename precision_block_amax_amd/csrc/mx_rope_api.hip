// mx_rope_api.hip -- the extern "C" entry points of the rotary positions and of
// the norm of each head (include/mx.h).  As in mx_api.hip: every argument is
// validated on the host before the first HIP call.
#include <math.h>

#include "mx_check.h"
#include "mx_rope_internal.h"

namespace {

using namespace mx;

constexpr int64_t kMaxTokens = (int64_t)1 << 31, kMaxHeads = (int64_t)1 << 16;

// Elements (token, head, 0 .. dim - 1) at token * lt + head * lh: tokens outermost or heads outermost, none of them
// twice.  Their bytes as one run of rows; n = -1 if they leave 64 bits, a status other than MX_OK for other strides.
mx_status_t heads_at(const void *p, int64_t tokens, int64_t heads, int64_t lt, int64_t lh, int64_t dim, Range *r) {
    *r = run(p, 0);
    if (tokens <= 0 || heads <= 0 || dim <= 0) return MX_OK;
    if (!p) return MX_ERR_INVALID_ARG;
    if (heads == 1) lh = dim;
    if (tokens == 1) lt = INT64_MAX;  // it has no stride
    if (lt < dim || lh < dim) return MX_ERR_INVALID_ARG;
    const Range token = rows_at(p, heads, lh, dim, 2);
    if (token.n >= 0 && token.n / 2 <= lt) {
        *r = rows_at(p, tokens, lt, token.n / 2, 2);
        return MX_OK;
    }
    const Range head = rows_at(p, tokens, lt, dim, 2);
    if (head.n < 0 || head.n / 2 > lh) return token.n < 0 && head.n < 0 ? ((*r = run(p, -1)), MX_OK) : MX_ERR_INVALID_ARG;
    *r = rows_at(p, heads, lh, head.n / 2, 2);
    return MX_OK;
}

mx_status_t check_common(const RopeArgs &a, int64_t q_heads, int64_t k_heads, int64_t dim, int64_t rot, int pos_type,
                         int layout) {
    if (q_heads < 0 || k_heads < 0 || a.tokens < 0 || dim < 0 || rot < 0 || rot > dim || rot % 2 != 0) return MX_ERR_INVALID_ARG;
    if (pos_type != MX_POS_I32 && pos_type != MX_POS_I64) return MX_ERR_INVALID_ARG;
    if (layout != MX_ROPE_HALF && layout != MX_ROPE_INTERLEAVED) return MX_ERR_INVALID_ARG;
    if (!isfinite(a.scale) || !(a.eps >= 0.0f) || isinf(a.eps)) return MX_ERR_INVALID_ARG;
    if (dim > kHeadMaxDim || a.tokens > kMaxTokens || q_heads > kMaxHeads || k_heads > kMaxHeads) return MX_ERR_UNSUPPORTED;
    return MX_OK;
}

// ranges: x, dy and out of both, positions, freqs, then `more` others; the outputs are checked against all
mx_status_t run_heads(RopeArgs &a, int op, int64_t dim, int64_t rot, int pos_type, int layout, const Range *more, int count,
                      void *stream) {
    Range r[16];
    int n = 0;
    mx_status_t st;
    const bool none = a.tokens == 0 || dim == 0;
    for (const HeadSet &h : a.s) {
        if ((st = heads_at(h.x, a.tokens, h.heads, h.xt, h.xh, dim, &r[n++])) != MX_OK) return st;
        if (op == NORM_ROPE_BWD && (st = heads_at(h.dy, a.tokens, h.heads, h.dt, h.dh, dim, &r[n++])) != MX_OK) return st;
        r[n++] = run(h.weight, h.weight ? dim * (a.param_bf16 ? 2 : 4) : 0);
    }
    const bool any = !none && a.s[0].heads + a.s[1].heads > 0;
    if (any && ((!a.pos && rot > 0) || (!a.freqs && rot > 0))) return MX_ERR_INVALID_ARG;
    r[n++] = run(a.pos, rot > 0 && any ? a.tokens * (pos_type == MX_POS_I64 ? 8 : 4) : 0);
    r[n++] = run(a.freqs, rot > 0 && any ? rot / 2 * 8 : 0);
    const int first = n;
    for (const HeadSet &h : a.s)
        if ((st = heads_at(h.out, a.tokens, h.heads, h.ot, h.oh, dim, &r[n++])) != MX_OK) return st;
    for (int i = 0; i < count; i++) r[n++] = more[i];
    if ((st = check_ranges(r, n, first)) != MX_OK) return st;
    if (!any && !(op == NORM_ROPE_BWD && dim > 0 && (a.s[0].dw || a.s[1].dw))) return MX_OK;
    if ((st = check_device()) != MX_OK) return st;
    a.dim = (int)dim;
    a.rot = (int)rot;
    a.pos64 = pos_type == MX_POS_I64;
    a.interleaved = layout == MX_ROPE_INTERLEAVED;
    return launched(launch_heads(a, op, (hipStream_t)stream));
}

HeadSet head_set(const void *x, int64_t xt, int64_t xh, int64_t heads, void *out, int64_t ot, int64_t oh) {
    HeadSet h{};
    h.x = (const uint16_t *)x;
    h.xt = xt;
    h.xh = xh;
    h.out = (uint16_t *)out;
    h.ot = ot;
    h.oh = oh;
    h.heads = (int)heads;
    return h;
}

}  // namespace

extern "C" {

mx_status_t mx_rope_frequencies(int64_t rot, double theta, mx_rope_scaling_t scaling, double factor, double low, double high,
                                double original, double *freqs) {
    const int k = raw(scaling);
    if (rot < 0 || rot % 2 != 0 || !(theta > 0) || !isfinite(theta) || k < MX_ROPE_PLAIN || k > MX_ROPE_BANDS)
        return MX_ERR_INVALID_ARG;
    if (k != MX_ROPE_PLAIN && (!(factor > 0) || !isfinite(factor))) return MX_ERR_INVALID_ARG;
    if (k == MX_ROPE_BANDS && (!(low >= 0) || !(high > low) || !isfinite(high) || !(original > 0) || !isfinite(original)))
        return MX_ERR_INVALID_ARG;
    if (rot > 0 && !freqs) return MX_ERR_INVALID_ARG;
    for (int64_t i = 0; i < rot / 2; i++) {
        double f = pow(theta, -2.0 * (double)i / (double)rot);
        if (k == MX_ROPE_LINEAR) f /= factor;
        if (k == MX_ROPE_BANDS) {
            const double turns = original * f / (2.0 * M_PI), keep = fmin(1.0, fmax(0.0, (turns - low) / (high - low)));
            f = f * keep + f / factor * (1.0 - keep);
        }
        freqs[i] = f;
    }
    return MX_OK;
}

mx_status_t mx_rope(const void *q_bf16, int64_t ldq, int64_t ldq_head, int64_t q_heads, const void *k_bf16, int64_t ldk,
                    int64_t ldk_head, int64_t k_heads, int64_t tokens, int64_t dim, const void *positions, mx_pos_t pos_type,
                    const double *freqs, int64_t rot, mx_rope_layout_t layout, float scale, int inverse, void *q_out,
                    int64_t ldqo, int64_t ldqo_head, void *k_out, int64_t ldko, int64_t ldko_head, void *stream) {
    RopeArgs a{};
    a.pos = positions;
    a.freqs = freqs;
    a.tokens = tokens;
    a.scale = scale;
    a.inverse = inverse != 0;
    const int p = raw(pos_type), l = raw(layout);
    if (inverse != 0 && inverse != 1) return MX_ERR_INVALID_ARG;
    const mx_status_t st = check_common(a, q_heads, k_heads, dim, rot, p, l);
    if (st != MX_OK) return st;
    a.s[0] = head_set(q_bf16, ldq, ldq_head, q_heads, q_out, ldqo, ldqo_head);
    a.s[1] = head_set(k_bf16, ldk, ldk_head, k_heads, k_out, ldko, ldko_head);
    return run_heads(a, ROPE, dim, rot, p, l, nullptr, 0, stream);
}

mx_status_t mx_qk_norm_rope(const void *q_bf16, int64_t ldq, int64_t ldq_head, int64_t q_heads, const void *k_bf16,
                            int64_t ldk, int64_t ldk_head, int64_t k_heads, int64_t tokens, int64_t dim,
                            const void *q_weight, const void *k_weight, mx_out_t param, float eps, const void *positions,
                            mx_pos_t pos_type, const double *freqs, int64_t rot, mx_rope_layout_t layout, float scale,
                            void *q_out, int64_t ldqo, int64_t ldqo_head, void *k_out, int64_t ldko, int64_t ldko_head,
                            void *stream) {
    RopeArgs a{};
    a.pos = positions;
    a.freqs = freqs;
    a.tokens = tokens;
    a.scale = scale;
    a.eps = eps;
    const int p = raw(pos_type), l = raw(layout), t = raw(param);
    if (t != MX_OUT_F32 && t != MX_OUT_BF16) return MX_ERR_INVALID_ARG;
    a.param_bf16 = t == MX_OUT_BF16;
    const mx_status_t st = check_common(a, q_heads, k_heads, dim, rot, p, l);
    if (st != MX_OK) return st;
    a.s[0] = head_set(q_bf16, ldq, ldq_head, q_heads, q_out, ldqo, ldqo_head);
    a.s[1] = head_set(k_bf16, ldk, ldk_head, k_heads, k_out, ldko, ldko_head);
    a.s[0].weight = q_weight;
    a.s[1].weight = k_weight;
    return run_heads(a, NORM_ROPE, dim, rot, p, l, nullptr, 0, stream);
}

int64_t mx_qk_norm_rope_backward_workspace(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim) {
    if (tokens <= 0 || q_heads < 0 || k_heads < 0 || dim <= 0 || dim > kHeadMaxDim) return 0;
    return heads_workspace(tokens, q_heads, k_heads, dim) * 4;
}

mx_status_t mx_qk_norm_rope_backward(const void *dq_bf16, int64_t lddq, int64_t lddq_head, const void *dk_bf16, int64_t lddk,
                                     int64_t lddk_head, const void *q_bf16, int64_t ldq, int64_t ldq_head, int64_t q_heads,
                                     const void *k_bf16, int64_t ldk, int64_t ldk_head, int64_t k_heads, int64_t tokens,
                                     int64_t dim, const void *q_weight, const void *k_weight, mx_out_t param, float eps,
                                     const void *positions, mx_pos_t pos_type, const double *freqs, int64_t rot,
                                     mx_rope_layout_t layout, float scale, void *dxq_bf16, int64_t lddxq, int64_t lddxq_head,
                                     void *dxk_bf16, int64_t lddxk, int64_t lddxk_head, float *dq_weight, float *dk_weight,
                                     void *workspace, int64_t workspace_bytes, void *stream) {
    RopeArgs a{};
    a.pos = positions;
    a.freqs = freqs;
    a.tokens = tokens;
    a.scale = scale;
    a.eps = eps;
    a.ws = (float *)workspace;
    const int p = raw(pos_type), l = raw(layout), t = raw(param);
    if (t != MX_OUT_F32 && t != MX_OUT_BF16) return MX_ERR_INVALID_ARG;
    a.param_bf16 = t == MX_OUT_BF16;
    const mx_status_t st = check_common(a, q_heads, k_heads, dim, rot, p, l);
    if (st != MX_OK) return st;
    a.s[0] = head_set(q_bf16, ldq, ldq_head, q_heads, dxq_bf16, lddxq, lddxq_head);
    a.s[1] = head_set(k_bf16, ldk, ldk_head, k_heads, dxk_bf16, lddxk, lddxk_head);
    a.s[0].weight = q_weight;
    a.s[1].weight = k_weight;
    a.s[0].dy = (const uint16_t *)dq_bf16;
    a.s[0].dt = lddq;
    a.s[0].dh = lddq_head;
    a.s[1].dy = (const uint16_t *)dk_bf16;
    a.s[1].dt = lddk;
    a.s[1].dh = lddk_head;
    a.s[0].dw = dq_weight;
    a.s[1].dw = dk_weight;
    const int64_t need = dq_weight || dk_weight ? mx_qk_norm_rope_backward_workspace(tokens, q_heads, k_heads, dim) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need || (uintptr_t)workspace % 16 != 0)) return MX_ERR_INVALID_ARG;
    const Range more[3] = {run(dq_weight, dq_weight ? dim * 4 : 0), run(dk_weight, dk_weight ? dim * 4 : 0), run(workspace, need)};
    return run_heads(a, NORM_ROPE_BWD, dim, rot, p, l, more, 3, stream);
}

}  // extern "C"
