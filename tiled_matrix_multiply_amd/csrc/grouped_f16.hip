// Grouped products of fp16 rows.
#include "grouped_mfma.hpp"

namespace tgemm {

hipError_t launch_grouped_f16(const GemmParams& p, const GroupArgs& ga, bool b_mn, int tile, int cus, hipStream_t s) {
  return launch_rows_type<F16, F16>(p, ga, b_mn, tile, cus, s);
}

}  // namespace tgemm
