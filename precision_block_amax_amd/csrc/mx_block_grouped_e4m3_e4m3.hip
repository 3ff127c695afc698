// mx_block_grouped_e4m3_e4m3.hip -- block-128 products by group for A in E4M3 and B in E4M3
#include "mx_block_gemm_kernels.h"

namespace mx {
hipError_t launch_block_gemm_grouped_0_0(const GroupedGemmArgs &g, bool bt, bool fp8_sums, hipStream_t s) {
    return launch_block_gemm_grouped_fmt<0, 0>(g, bt, fp8_sums, s);
}
}  // namespace mx
