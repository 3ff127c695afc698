// mx_block_gemm_e5m2_e5m2.hip -- block-128 product kernels for A in E5M2 and B in E5M2
#include "mx_block_gemm_kernels.h"

namespace mx {
hipError_t launch_block_gemm_1_1(const BlockGemmArgs &g, bool bt, bool fp8_sums, hipStream_t s) {
    return launch_block_gemm_fmt<1, 1>(g, bt, fp8_sums, s);
}
}  // namespace mx
