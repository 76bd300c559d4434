// The matrix products in bf16 (templates: blk_gemm.hpp).
#include "blk_gemm.hpp"

namespace blk {
rr_status_t launch_gemm_bf16(const GemmArgs& a, const GemmPlan& p, hipStream_t s) {
    return launch_gemm<bf16>(a, p, s);
}
}  // namespace blk
