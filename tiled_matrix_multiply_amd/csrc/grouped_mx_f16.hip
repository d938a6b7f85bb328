// Products by expert in MXFP4 with a result in fp16.
#include "grouped_mfma.hpp"

namespace tgemm {

hipError_t launch_grouped_mx_f16(const GemmParams& p, const GroupArgs& ga, int tile, int cus, hipStream_t s) {
  return launch_mx_type<F16>(p, ga, tile, cus, s);
}

}  // namespace tgemm
