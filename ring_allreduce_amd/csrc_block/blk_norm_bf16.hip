// The norms over rows of bf16 (templates: blk_norm.hpp).
#include "blk_norm.hpp"

namespace blk {
void launch_norm_bf16(const NormArgs& a, const Config& c, unsigned grid, bool back, hipStream_t s) {
    launch_rows<bf16>(a, c, grid, back, s);
}
}  // namespace blk
