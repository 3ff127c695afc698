// mx_rope_internal.h -- launchers of the rotary positions and of the norm of
// each head.  Not part of the public ABI.
#pragma once
#include "mx_internal.h"

namespace mx {

constexpr int kHeadMaxDim = 512;  // a head is held in the registers of one wave

// the heads of one tensor, element (token, head, i) at token * t + head * h + i of each array
struct HeadSet {
    const uint16_t *x, *dy;  // dy: backward only
    uint16_t *out;           // y, or dx
    int64_t xt, xh, dt, dh, ot, oh;
    const void *weight;      // may be nullptr
    float *dw;               // backward; may be nullptr
    int heads;
};

struct RopeArgs {
    HeadSet s[2];  // queries, keys
    const void *pos;
    const double *freqs;  // rot / 2 of them
    float *ws;
    int64_t tokens;
    int dim, rot;
    float scale, eps;
    bool pos64, interleaved, inverse, param_bf16;
};

enum HeadOp : int { ROPE = 0, NORM_ROPE = 1, NORM_ROPE_BWD = 2 };

// tokens > 0 and some heads
hipError_t launch_heads(const RopeArgs &a, int op, hipStream_t stream);
// floats of workspace that NORM_ROPE_BWD uses where a gradient of a weight is wanted
int64_t heads_workspace(int64_t tokens, int64_t heads_q, int64_t heads_k, int64_t dim);

}  // namespace mx
