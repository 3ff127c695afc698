// mx_block_grouped_e5m2_e4m3.hip -- block-128 products by group for A in E5M2 and B in E4M3
#include "mx_block_gemm_kernels.h"

namespace mx {
hipError_t launch_block_gemm_grouped_1_0(const GroupedGemmArgs &g, bool bt, bool fp8_sums, hipStream_t s) {
    return launch_block_gemm_grouped_fmt<1, 0>(g, bt, fp8_sums, s);
}
}  // namespace mx
