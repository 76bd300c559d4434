// The gated products in bf16 (templates: blk_gated.hpp).
#include "blk_gated.hpp"

namespace blk {
rr_status_t launch_gated_bf16(const GemmArgs& a, const GemmPlan& p, hipStream_t s) {
    return launch_gated<bf16>(a, p, s);
}
}  // namespace blk
