// Grouped weight gradients of bf16 rows.
#include "grouped_mfma.hpp"

namespace tgemm {

hipError_t launch_grouped_wgrad_bf16(const GemmParams& p, const GroupArgs& ga, const BiasGrad& b, int c_type,
                                   int tile, hipStream_t s) {
  return c_type == F32 ? launch_wgrad_type<BF16, F32>(p, ga, b, tile, s)
                       : launch_wgrad_type<BF16, BF16>(p, ga, b, tile, s);
}

}  // namespace tgemm
