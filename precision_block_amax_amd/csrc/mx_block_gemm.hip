// mx_block_gemm.hip -- dispatch of mx_block_gemm to the kernels of
// mx_block_gemm_kernels.h; each operand-format pair is a translation unit of
// its own (mx_block_gemm_<fa>_<fb>.hip), so the library builds in parallel.
#include "mx_block_gemm_kernels.h"

namespace mx {

#define MX_PAIR(fa, fb) hipError_t launch_block_gemm_##fa##_##fb(const BlockGemmArgs &g, bool bt, bool fp8_sums, hipStream_t s);
MX_PAIR(0, 0) MX_PAIR(0, 1) MX_PAIR(1, 0) MX_PAIR(1, 1)
#undef MX_PAIR

hipError_t launch_block_gemm(const BlockGemmArgs &g, int fa, int fb, bool bt, bool fp8_sums, hipStream_t s) {
    if (g.K == 0) {
        // 256 elements per workgroup, at most 2^31 of them per launch
        const int64_t rows = ((int64_t)1 << 31) / g.N > 0 ? ((int64_t)1 << 31) / g.N : 1;
        for (int64_t m = 0; m < g.M; m += rows) {
            const int mr = (int)min(rows, (int64_t)g.M - m);
            const dim3 grid((unsigned)(((int64_t)mr * g.N + 255) / 256));
            uint8_t *c = (uint8_t *)g.c + m * g.ldc * (g.c_bf16 ? 2 : 4);
            if (g.c_bf16) hipLaunchKernelGGL((k_zero<true>), grid, dim3(256), 0, s, (void *)c, g.ldc, mr, g.N);
            else hipLaunchKernelGGL((k_zero<false>), grid, dim3(256), 0, s, (void *)c, g.ldc, mr, g.N);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    switch (fa * 2 + fb) {
    case 0: return launch_block_gemm_0_0(g, bt, fp8_sums, s);
    case 1: return launch_block_gemm_0_1(g, bt, fp8_sums, s);
    case 2: return launch_block_gemm_1_0(g, bt, fp8_sums, s);
    default: return launch_block_gemm_1_1(g, bt, fp8_sums, s);
    }
}

}  // namespace mx
