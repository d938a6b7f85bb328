// Products of 8-bit integers, single and grouped, with a result in fp16.
#include "grouped_mfma.hpp"

namespace tgemm {

hipError_t launch_grouped_i8_f16(const GemmParams& p, const GroupArgs& ga, bool b_mn, int tile, int cus, hipStream_t s) {
  return launch_rows_type<I8, F16>(p, ga, b_mn, tile, cus, s);
}

}  // namespace tgemm
