// The norms over rows of f32 (templates: blk_norm.hpp).
#include "blk_norm.hpp"

namespace blk {
void launch_norm_f32(const NormArgs& a, const Config& c, unsigned grid, bool back, hipStream_t s) {
    launch_rows<float>(a, c, grid, back, s);
}
}  // namespace blk
