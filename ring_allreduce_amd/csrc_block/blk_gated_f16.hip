// The gated products in fp16 (templates: blk_gated.hpp).
#include "blk_gated.hpp"

namespace blk {
rr_status_t launch_gated_f16(const GemmArgs& a, const GemmPlan& p, hipStream_t s) {
    return launch_gated<f16>(a, p, s);
}
}  // namespace blk
