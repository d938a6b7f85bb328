// Host side of the entry points declared in include/gemm_grouped.h: argument validation, kernel
// choice and launches.  Nothing is allocated per call and the offsets are never read here.
#include "gemm_grouped.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grouped.hpp"
#include "handle.hpp"

namespace tgemm {
hipError_t launch_grouped_any(const GemmParams& p, const GroupArgs& ga, int type, int c_type, bool b_mn,
                              hipStream_t s);
hipError_t launch_grouped_wgrad_any(const GemmParams& p, const GroupArgs& ga, int type, int c_type,
                                    hipStream_t s);
hipError_t launch_bias_grad(const void* D, int64_t ldd, int M, int N, int type, const GroupArgs& ga,
                            float* dbias, hipStream_t s);
hipError_t launch_quantize_rows(const void* X, int64_t ldx, int M, int K, int x_type, int8_t* Q, int64_t ldq,
                                float* scales, hipStream_t s);
}  // namespace tgemm

namespace {

constexpr int64_t kMaxDim = 0x7fffffff;
constexpr int64_t kMaxGroups = 65535;
constexpr int64_t kMaxK8 = 131071;  // 128 * 128 * K < 2^31

// What the products and the gradient have in common: three matrices, some of them per group.
struct GArgs {
  bool wgrad, i8;
  int64_t groups;
  const int64_t* offsets;
  int64_t M, N, K;
  int transB;
  const void* A;
  int64_t lda;
  const float* sa;
  const void* B;  // the weights; for the gradient D
  int64_t ldb, stride_b;
  const float* sb;
  const void* C;
  int64_t ldc, stride_c;
  gemm_dtype_t at, ct;
  uint32_t epi;
  const float* bias;  // read; for the gradient dbias, written
};

int es(gemm_dtype_t t) { return t == GEMM_F32 ? 4 : t == GEMM_F16 || t == GEMM_BF16 ? 2 : 0; }

struct Range {
  __int128 lo, hi;
};
// Byte range of `count` matrices of rows x cols elements of `size` bytes, `stride` elements apart.
Range range(const void* p, int64_t rows, int64_t cols, int64_t ld, int size, int64_t count = 1, int64_t stride = 0) {
  const __int128 lo = (__int128)(uintptr_t)p;
  if (!p || rows <= 0 || cols <= 0 || count <= 0) return {lo, lo};
  return {lo, lo + ((__int128)(count - 1) * stride + (__int128)(rows - 1) * ld + cols) * size};
}
bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }
bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

gemm_status_t check(const GArgs& a) {
  if (a.M < 0 || a.N < 0 || a.K < 0 || a.groups < 0) return GEMM_ERR_INVALID_VALUE;
  if (a.transB != 0 && a.transB != 1) return GEMM_ERR_INVALID_VALUE;
  if (a.epi & ~(GEMM_EPI_BIAS | GEMM_EPI_GELU)) return GEMM_ERR_INVALID_VALUE;
  if (a.i8) {
    if (!es(a.ct)) return GEMM_ERR_UNSUPPORTED;
    if (a.K > kMaxK8) return GEMM_ERR_UNSUPPORTED;
  } else {
    if (a.at != GEMM_F16 && a.at != GEMM_BF16) return GEMM_ERR_UNSUPPORTED;
    if (a.ct != a.at && !(a.wgrad && a.ct == GEMM_F32)) return GEMM_ERR_UNSUPPORTED;
  }
  if (a.M > kMaxDim || a.N > kMaxDim || a.K > kMaxDim || a.groups > kMaxGroups) return GEMM_ERR_UNSUPPORTED;
  if (a.N == 0 || a.groups == 0) return GEMM_OK;                        // nothing to compute
  if (a.wgrad ? (a.K == 0 && !a.bias) : a.M == 0) return GEMM_OK;
  if (!a.offsets && !(a.i8 && a.groups == 1)) return GEMM_ERR_INVALID_VALUE;
  if (!aligned(a.offsets, 8)) return GEMM_ERR_INVALID_VALUE;
  const int in = a.i8 ? 1 : es(a.at), out = es(a.ct);
  const Range off = range(a.offsets, 1, a.groups + 1, 0, 8);
  if (a.wgrad) {
    const int64_t rows = a.transB ? a.N : a.K, cols = a.transB ? a.K : a.N;
    if (a.K > 0) {
      if (!a.C || a.ldc < cols) return GEMM_ERR_INVALID_VALUE;
      if (a.groups > 1 && (__int128)a.stride_c < (__int128)(rows - 1) * a.ldc + cols) return GEMM_ERR_INVALID_VALUE;
    }
    if (a.M > 0) {
      if (a.K > 0 && (!a.A || a.lda < a.K)) return GEMM_ERR_INVALID_VALUE;
      if (!a.B || a.ldb < a.N) return GEMM_ERR_INVALID_VALUE;
    }
    const Range rc = a.K > 0 ? range(a.C, rows, cols, a.ldc, out, a.groups, a.stride_c) : Range{0, 0};
    const Range ra = range(a.A, a.M, a.K, a.lda, in), rd = range(a.B, a.M, a.N, a.ldb, in);
    const Range rb = range(a.bias, 1, a.groups * a.N, 0, 4);
    if (overlaps(rc, ra) || overlaps(rc, rd) || overlaps(rc, off) || overlaps(rc, rb) || overlaps(rb, ra) ||
        overlaps(rb, rd) || overlaps(rb, off))
      return GEMM_ERR_ALIAS;
    return GEMM_OK;
  }
  if (!a.C || a.ldc < a.N) return GEMM_ERR_INVALID_VALUE;
  if ((a.epi & GEMM_EPI_BIAS) && !a.bias) return GEMM_ERR_INVALID_VALUE;
  if (a.stride_b < 0) return GEMM_ERR_INVALID_VALUE;
  if (a.i8 && (!a.sa || !a.sb)) return GEMM_ERR_INVALID_VALUE;
  const Range rc = range(a.C, a.M, a.N, a.ldc, out);
  if (a.K > 0) {
    const int64_t rows = a.transB ? a.N : a.K, cols = a.transB ? a.K : a.N;
    if (!a.A || !a.B || a.lda < a.K || a.ldb < cols) return GEMM_ERR_INVALID_VALUE;
    if (overlaps(rc, range(a.A, a.M, a.K, a.lda, in)) ||
        overlaps(rc, range(a.B, rows, cols, a.ldb, in, a.groups, a.stride_b)))
      return GEMM_ERR_ALIAS;
  }
  if (overlaps(rc, off)) return GEMM_ERR_ALIAS;
  if ((a.epi & GEMM_EPI_BIAS) && overlaps(rc, range(a.bias, 1, a.groups * a.N, 0, 4))) return GEMM_ERR_ALIAS;
  if (a.i8 && (overlaps(rc, range(a.sa, 1, a.M, 0, 4)) || overlaps(rc, range(a.sb, 1, a.groups * a.N, 0, 4))))
    return GEMM_ERR_ALIAS;
  return GEMM_OK;
}

tgemm::GemmParams params(const GArgs& a, float alpha, float beta, void* C) {
  tgemm::GemmParams p{};
  p.A = a.A;
  p.B = a.B;
  p.C = C;
  p.lda = a.lda;
  p.ldb = a.ldb;
  p.ldc = a.ldc;
  p.M = (int)a.M;
  p.N = (int)a.N;
  p.K = (int)a.K;
  p.alpha = alpha;
  p.beta = beta;
  p.epi = a.epi;
  return p;
}

bool valid(gemm_handle_t h) { return h && h->magic == tgemm::kHandleMagic; }

gemm_status_t status(hipError_t e) { return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH; }

// Tiles of 64 x 64, the smallest, must be countable in 31 bits.
bool countable(int64_t row_tiles, int64_t n) { return (__int128)row_tiles * ((n + 63) / 64) <= kMaxDim; }

gemm_status_t run_rows(gemm_handle_t h, gemm_grouped_kernel_t kernel, void* stream, const GArgs& a, float alpha,
                       float beta, void* C) {
  if (!valid(h)) return GEMM_ERR_INVALID_HANDLE;
  const gemm_status_t st = check(a);
  if (st != GEMM_OK) return st;
  if (a.M == 0 || a.N == 0 || a.groups == 0) return GEMM_OK;
  if (!countable(tgemm::max_row_tiles(a.M, a.groups, 64), a.N)) return GEMM_ERR_UNSUPPORTED;
  if (kernel != GEMM_GROUPED_AUTO && kernel != GEMM_GROUPED_ANY) return GEMM_ERR_INVALID_VALUE;
  tgemm::GemmParams p = params(a, alpha, beta, C);
  p.bias = (a.epi & GEMM_EPI_BIAS) ? a.bias : nullptr;
  p.ra = a.sa;
  p.rb = a.sb;
  const tgemm::GroupArgs ga{a.offsets, (int)a.groups, a.stride_b, 0};
  const int type = a.i8 ? tgemm::I8 : (int)a.at;
  tgemm::DeviceGuard g(h->device);
  return status(tgemm::launch_grouped_any(p, ga, type, a.ct, a.transB == 0, static_cast<hipStream_t>(stream)));
}

gemm_status_t run_wgrad(gemm_handle_t h, gemm_grouped_kernel_t kernel, void* stream, const GArgs& a, float alpha,
                        float beta, void* C, float* dbias) {
  if (!valid(h)) return GEMM_ERR_INVALID_HANDLE;
  const gemm_status_t st = check(a);
  if (st != GEMM_OK) return st;
  if (a.N == 0 || a.groups == 0 || (a.K == 0 && !dbias)) return GEMM_OK;
  if (kernel != GEMM_GROUPED_AUTO && kernel != GEMM_GROUPED_ANY) return GEMM_ERR_INVALID_VALUE;
  const tgemm::GroupArgs ga{a.offsets, (int)a.groups, 0, a.stride_c};
  // The kernels compute C = X^T Y: stored N x K, the gradient is D^T A.
  tgemm::GemmParams p = params(a, alpha, beta, C);
  p.A = a.transB ? a.B : a.A;
  p.lda = a.transB ? a.ldb : a.lda;
  p.B = a.transB ? a.A : a.B;
  p.ldb = a.transB ? a.lda : a.ldb;
  p.M = (int)(a.transB ? a.N : a.K);
  p.N = (int)(a.transB ? a.K : a.N);
  p.K = (int)a.M;
  p.epi = 0;
  if (!countable(((int64_t)p.M + 63) / 64 * a.groups, p.N)) return GEMM_ERR_UNSUPPORTED;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  tgemm::DeviceGuard g(h->device);
  if (dbias) {
    const hipError_t e = tgemm::launch_bias_grad(a.B, a.ldb, (int)a.M, (int)a.N, a.at, ga, dbias, s);
    if (e != hipSuccess) return GEMM_ERR_LAUNCH;
  }
  if (a.K == 0) return GEMM_OK;
  return status(tgemm::launch_grouped_wgrad_any(p, ga, a.at, a.ct, s));
}

gemm_status_t check_quantize(int64_t M, int64_t K, const void* X, int64_t ldx, gemm_dtype_t xt, const void* Q,
                             int64_t ldq, const float* scales) {
  if (M < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
  if (!es(xt) || M > kMaxDim || K > kMaxDim) return GEMM_ERR_UNSUPPORTED;
  if (M == 0) return GEMM_OK;
  if (!scales) return GEMM_ERR_INVALID_VALUE;
  if (K > 0 && (!X || !Q || ldx < K || ldq < K)) return GEMM_ERR_INVALID_VALUE;
  const Range rx = range(X, M, K, ldx, es(xt)), rq = range(Q, M, K, ldq, 1), rs = range(scales, 1, M, 0, 4);
  if (overlaps(rq, rx) || overlaps(rs, rx) || overlaps(rs, rq)) return GEMM_ERR_ALIAS;
  return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status_t gemm_check_args_grouped(int64_t groups, const int64_t* offsets, int64_t M, int64_t N, int64_t K,
                                      int transB, const void* A, int64_t lda, const float* sa, const void* B,
                                      int64_t ldb, int64_t stride_b, const float* sb, const void* C,
                                      int64_t ldc, int i8, gemm_dtype_t type, gemm_dtype_t c_type,
                                      uint32_t epilogue, const float* bias) {
  return check(GArgs{false, i8 != 0, groups, offsets, M, N, K, transB, A, lda, sa, B, ldb, stride_b, sb, C, ldc, 0,
                     type, c_type, epilogue, bias});
}

gemm_status_t gemm_run_grouped(gemm_handle_t h, gemm_grouped_kernel_t kernel, void* stream, int64_t groups,
                               const int64_t* offsets, int64_t M, int64_t N, int64_t K, int transB, float alpha,
                               const void* A, int64_t lda, const void* B, int64_t ldb, int64_t stride_b,
                               float beta, void* C, int64_t ldc, gemm_dtype_t type, uint32_t epilogue,
                               const float* bias) {
  const GArgs a{false, false, groups, offsets, M, N, K, transB, A, lda, nullptr, B, ldb, stride_b, nullptr, C, ldc, 0,
                type, type, epilogue, bias};
  return run_rows(h, kernel, stream, a, alpha, beta, C);
}

gemm_status_t gemm_run_i8(gemm_handle_t h, gemm_grouped_kernel_t kernel, void* stream, int64_t M, int64_t N,
                          int64_t K, int transB, float alpha, const int8_t* A, int64_t lda, const float* sa,
                          const int8_t* B, int64_t ldb, const float* sb, float beta, void* C, int64_t ldc,
                          gemm_dtype_t c_type, uint32_t epilogue, const float* bias) {
  const GArgs a{false, true, 1, nullptr, M, N, K, transB, A, lda, sa, B, ldb, 0, sb, C, ldc, 0, c_type, c_type,
                epilogue, bias};
  return run_rows(h, kernel, stream, a, alpha, beta, C);
}

gemm_status_t gemm_run_grouped_i8(gemm_handle_t h, gemm_grouped_kernel_t kernel, void* stream, int64_t groups,
                                  const int64_t* offsets, int64_t M, int64_t N, int64_t K, int transB,
                                  float alpha, const int8_t* A, int64_t lda, const float* sa, const int8_t* B,
                                  int64_t ldb, int64_t stride_b, const float* sb, float beta, void* C,
                                  int64_t ldc, gemm_dtype_t c_type, uint32_t epilogue, const float* bias) {
  if (groups > 0 && M > 0 && N > 0 && !offsets) return valid(h) ? GEMM_ERR_INVALID_VALUE : GEMM_ERR_INVALID_HANDLE;
  const GArgs a{false, true, groups, offsets, M, N, K, transB, A, lda, sa, B, ldb, stride_b, sb, C, ldc, 0, c_type,
                c_type, epilogue, bias};
  return run_rows(h, kernel, stream, a, alpha, beta, C);
}

gemm_status_t gemm_check_args_grouped_wgrad(int64_t groups, const int64_t* offsets, int64_t M, int64_t N,
                                            int64_t K, int transB, const void* A, int64_t lda, const void* D,
                                            int64_t ldd, const void* C, int64_t ldc, int64_t stride_c,
                                            gemm_dtype_t type, gemm_dtype_t c_type, const float* dbias) {
  return check(GArgs{true, false, groups, offsets, M, N, K, transB, A, lda, nullptr, D, ldd, 0, nullptr, C, ldc, stride_c,
                     type, c_type, 0, dbias});
}

gemm_status_t gemm_run_grouped_wgrad(gemm_handle_t h, gemm_grouped_kernel_t kernel, void* stream, int64_t groups,
                                     const int64_t* offsets, int64_t M, int64_t N, int64_t K, int transB,
                                     float alpha, const void* A, int64_t lda, const void* D, int64_t ldd,
                                     float beta, void* C, int64_t ldc, int64_t stride_c, gemm_dtype_t type,
                                     gemm_dtype_t c_type, float* dbias) {
  const GArgs a{true, false, groups, offsets, M, N, K, transB, A, lda, nullptr, D, ldd, 0, nullptr, C, ldc, stride_c,
                type, c_type, 0, dbias};
  return run_wgrad(h, kernel, stream, a, alpha, beta, C, dbias);
}

gemm_status_t gemm_check_args_quantize_rows(int64_t M, int64_t K, const void* X, int64_t ldx,
                                            gemm_dtype_t x_type, const int8_t* Q, int64_t ldq,
                                            const float* scales) {
  return check_quantize(M, K, X, ldx, x_type, Q, ldq, scales);
}

gemm_status_t gemm_quantize_rows(gemm_handle_t h, void* stream, int64_t M, int64_t K, const void* X, int64_t ldx,
                                 gemm_dtype_t x_type, int8_t* Q, int64_t ldq, float* scales) {
  if (!valid(h)) return GEMM_ERR_INVALID_HANDLE;
  const gemm_status_t st = check_quantize(M, K, X, ldx, x_type, Q, ldq, scales);
  if (st != GEMM_OK) return st;
  if (M == 0) return GEMM_OK;
  tgemm::DeviceGuard g(h->device);
  return status(tgemm::launch_quantize_rows(X, ldx, (int)M, (int)K, x_type, Q, ldq, scales,
                                            static_cast<hipStream_t>(stream)));
}

}  // extern "C"
