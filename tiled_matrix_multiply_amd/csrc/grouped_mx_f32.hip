// Products by expert in MXFP4 with a result in fp32.
#include "grouped_mfma.hpp"

namespace tgemm {

hipError_t launch_grouped_mx_f32(const GemmParams& p, const GroupArgs& ga, int tile, int cus, hipStream_t s) {
  return launch_mx_type<F32>(p, ga, tile, cus, s);
}

}  // namespace tgemm
