// Products by expert in MXFP4 with a result in bf16.
#include "grouped_mfma.hpp"

namespace tgemm {

hipError_t launch_grouped_mx_bf16(const GemmParams& p, const GroupArgs& ga, int tile, int cus, hipStream_t s) {
  return launch_mx_type<BF16>(p, ga, tile, cus, s);
}

}  // namespace tgemm
