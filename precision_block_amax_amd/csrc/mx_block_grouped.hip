// mx_block_grouped.hip -- dispatch of mx_block_gemm_grouped and
// mx_block_gemm_grouped_k to the kernels of mx_block_gemm_kernels.h; each
// operand-format pair of either is a translation unit of its own.
#include "mx_block_gemm_kernels.h"

namespace mx {

#define MX_PAIR(fa, fb)                                                                                                  \
    hipError_t launch_block_gemm_grouped_##fa##_##fb(const GroupedGemmArgs &g, bool bt, bool fp8_sums, hipStream_t s);   \
    hipError_t launch_block_gemm_grouped_k_##fa##_##fb(const GroupedGemmArgs &g, bool fp8_sums, hipStream_t s);
MX_PAIR(0, 0) MX_PAIR(0, 1) MX_PAIR(1, 0) MX_PAIR(1, 1)
#undef MX_PAIR

namespace {
// C's rows of groups = 0 (K == 0)
template <bool BF16OUT>
__global__ __launch_bounds__(256) void k_zero_rows(GroupedGemmArgs g) {
    GroupChunk<1> chunk;
    const int rows = group_units(chunk, g.ends, g.groups, g.rows);  // groups lie side by side from row 0 on
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)rows * g.N; i += step) {
        const int64_t at = i / g.N * g.ldc + i % g.N;
        if (BF16OUT) reinterpret_cast<uint16_t *>(g.c)[at] = 0;
        else reinterpret_cast<float *>(g.c)[at] = 0.f;
    }
}
}  // namespace

hipError_t launch_block_gemm_grouped(const GroupedGemmArgs &g, int fa, int fb, bool bt, bool fp8_sums, hipStream_t s) {
    if (g.K == 0) {
        if (g.c_bf16) hipLaunchKernelGGL((k_zero_rows<true>), dim3(1024), dim3(256), 0, s, g);
        else hipLaunchKernelGGL((k_zero_rows<false>), dim3(1024), dim3(256), 0, s, g);
        return hipGetLastError();
    }
    switch (fa * 2 + fb) {
    case 0: return launch_block_gemm_grouped_0_0(g, bt, fp8_sums, s);
    case 1: return launch_block_gemm_grouped_0_1(g, bt, fp8_sums, s);
    case 2: return launch_block_gemm_grouped_1_0(g, bt, fp8_sums, s);
    default: return launch_block_gemm_grouped_1_1(g, bt, fp8_sums, s);
    }
}

hipError_t launch_block_gemm_grouped_k(const GroupedGemmArgs &g, int fa, int fb, bool fp8_sums, hipStream_t s) {
    switch (fa * 2 + fb) {
    case 0: return launch_block_gemm_grouped_k_0_0(g, fp8_sums, s);
    case 1: return launch_block_gemm_grouped_k_0_1(g, fp8_sums, s);
    case 2: return launch_block_gemm_grouped_k_1_0(g, fp8_sums, s);
    default: return launch_block_gemm_grouped_k_1_1(g, fp8_sums, s);
    }
}

}  // namespace mx
