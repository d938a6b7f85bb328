// Argument checks that the host sides of the entry points share.
#pragma once

#include <stdint.h>

#include "handle.hpp"

namespace tgemm {
namespace checks {

constexpr int64_t kMaxDim = 0x7fffffff - 1023;      // tile edges past a dimension still fit 31 bits
constexpr int64_t kMaxRowBytes = int64_t(1) << 23;  // the kernels' 32-bit lane offsets span up to 256 rows

inline int es(gemm_dtype_t t) { return t == GEMM_F32 ? 4 : t == GEMM_F16 || t == GEMM_BF16 ? 2 : 0; }

struct Range {
  __int128 lo, hi;
};
// Byte range of `count` matrices of rows x cols elements of `size` bytes, `stride` elements apart.
inline Range range(const void* p, int64_t rows, int64_t cols, int64_t ld, int size, int64_t count = 1, int64_t stride = 0) {
  const __int128 lo = (__int128)(uintptr_t)p;
  if (!p || rows <= 0 || cols <= 0 || count <= 0) return {lo, lo};
  return {lo, lo + ((__int128)(count - 1) * stride + (__int128)(rows - 1) * ld + cols) * size};
}
inline bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }
inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool valid(gemm_handle_t h) { return h && h->magic == kHandleMagic; }
inline gemm_status_t status(hipError_t e) { return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH; }

}  // namespace checks
}  // namespace tgemm
