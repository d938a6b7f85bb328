// Products of 8-bit integers, single and grouped, with a result in bf16.
#include "grouped_mfma.hpp"

namespace tgemm {

hipError_t launch_grouped_i8_bf16(const GemmParams& p, const GroupArgs& ga, bool b_mn, int tile, int cus, hipStream_t s) {
  return launch_rows_type<I8, BF16>(p, ga, b_mn, tile, cus, s);
}

}  // namespace tgemm
