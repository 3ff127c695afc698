// mx_block_grouped_k_e4m3_e5m2.hip -- block-128 products by group along K for A in E4M3 and B in E5M2
#include "mx_block_gemm_kernels.h"

namespace mx {
hipError_t launch_block_gemm_grouped_k_0_1(const GroupedGemmArgs &g, bool fp8_sums, hipStream_t s) {
    return launch_block_gemm_grouped_k_fmt<0, 1>(g, fp8_sums, s);
}
}  // namespace mx
