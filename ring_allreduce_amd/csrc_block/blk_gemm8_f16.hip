// The products of 8-bit operands with results in fp16 (templates: blk_gemm8.hpp).
#include "blk_gemm8.hpp"

namespace blk {
rr_status_t launch_gemm8_f16(const GemmArgs& a, const GemmPlan& p, hipStream_t s) {
    return launch_gemm8<f16, false>(a, p, s);
}
rr_status_t launch_gated8_f16(const GemmArgs& a, const GemmPlan& p, hipStream_t s) {
    return launch_gemm8<f16, true>(a, p, s);
}
}  // namespace blk
