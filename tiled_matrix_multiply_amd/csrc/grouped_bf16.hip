// Grouped products of bf16 rows.
#include "grouped_mfma.hpp"

namespace tgemm {

hipError_t launch_grouped_bf16(const GemmParams& p, const GroupArgs& ga, bool b_mn, int tile, int cus, hipStream_t s) {
  return launch_rows_type<BF16, BF16>(p, ga, b_mn, tile, cus, s);
}

}  // namespace tgemm
