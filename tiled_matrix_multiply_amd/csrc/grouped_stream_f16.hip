// Products for few rows per group, f16 rows.
#include "grouped_stream.hpp"

namespace tgemm {

hipError_t launch_stream_f16(const GemmParams& p, const GroupArgs& ga, int c_type, bool kn, int rows, int waves,
                            hipStream_t s) {
  return launch_stream_type<F16>(p, ga, c_type, kn, rows, waves, s);
}

}  // namespace tgemm
