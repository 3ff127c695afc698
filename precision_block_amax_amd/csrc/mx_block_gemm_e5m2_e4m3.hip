// mx_block_gemm_e5m2_e4m3.hip -- block-128 product kernels for A in E5M2 and B in E4M3
#include "mx_block_gemm_kernels.h"

namespace mx {
hipError_t launch_block_gemm_1_0(const BlockGemmArgs &g, bool bt, bool fp8_sums, hipStream_t s) {
    return launch_block_gemm_fmt<1, 0>(g, bt, fp8_sums, s);
}
}  // namespace mx
