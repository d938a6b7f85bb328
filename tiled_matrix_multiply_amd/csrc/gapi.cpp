// Host side of the entry points declared in include/gemm_grouped.h: argument validation, kernel
// choice and launches.  Nothing is allocated per call and the offsets are never read here.
#include "gemm_grouped.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grouped.hpp"
#include "handle.hpp"

namespace tgemm {
// grouped_mfma.hpp's tiles (its GroupedTile numbers; 0: any alignment)
hipError_t launch_grouped_f16(const GemmParams&, const GroupArgs&, bool b_mn, int tile, int cus, hipStream_t);
hipError_t launch_grouped_bf16(const GemmParams&, const GroupArgs&, bool b_mn, int tile, int cus, hipStream_t);
hipError_t launch_grouped_i8_f16(const GemmParams&, const GroupArgs&, bool b_mn, int tile, int cus, hipStream_t);
hipError_t launch_grouped_i8_bf16(const GemmParams&, const GroupArgs&, bool b_mn, int tile, int cus, hipStream_t);
hipError_t launch_grouped_i8_f32(const GemmParams&, const GroupArgs&, bool b_mn, int tile, int cus, hipStream_t);
hipError_t launch_grouped_wgrad_f16(const GemmParams&, const GroupArgs&, const BiasGrad&, int c_type, int tile,
                                    hipStream_t);
hipError_t launch_grouped_wgrad_bf16(const GemmParams&, const GroupArgs&, const BiasGrad&, int c_type, int tile,
                                     hipStream_t);
hipError_t launch_stream_f16(const GemmParams&, const GroupArgs&, int c_type, bool kn, int rows, int waves, hipStream_t);
hipError_t launch_stream_bf16(const GemmParams&, const GroupArgs&, int c_type, bool kn, int rows, int waves, hipStream_t);
hipError_t launch_stream_i8(const GemmParams&, const GroupArgs&, int c_type, bool kn, int rows, int waves, hipStream_t);
hipError_t launch_quantize_rows(const void* X, int64_t ldx, int M, int K, int x_type, int8_t* Q, int64_t ldq,
                                float* scales, hipStream_t s);
}  // namespace tgemm

namespace {

constexpr int64_t kMaxDim = 0x7fffffff - 1023;  // tile edges past a dimension still fit 31 bits
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

// Workgroups must be countable in 31 bits, with the worst case's row tiles and a last round of 8.
// (Dimensions near 2^31 and many groups pass 63 bits together, hence the 128.)
bool countable(__int128 row_tiles, int64_t n, int64_t bn) { return row_tiles * ((n + bn - 1) / bn) <= kMaxDim - 16; }

// The same of a whole call, in the smallest tiles that any alignment and size can take: 64 x 64.
bool countable(const GArgs& a) {
  if (!a.wgrad) return countable(tgemm::max_row_tiles(a.M, a.groups, 64), a.N, 64);
  const int64_t rows = a.transB ? a.N : a.K, cols = a.transB ? a.K : a.N;
  const __int128 tiles = (__int128)((rows + 63) / 64) * ((cols + 63) / 64 + 7);  // a group's, with a last round of 8
  return countable(((a.N + 63) / 64 + tiles) * a.groups, 1, 1);                  // and its bias gradient's columns
}

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
  if (!countable(a)) return GEMM_ERR_UNSUPPORTED;
  if (!a.offsets && !(a.i8 && a.groups == 1)) return GEMM_ERR_INVALID_VALUE;
  if (!aligned(a.offsets, 8)) return GEMM_ERR_INVALID_VALUE;
  const int in = a.i8 ? 1 : es(a.at), out = es(a.ct);
  const Range off = range(a.offsets, 1, a.groups + 1, 0, 8);
  if (a.wgrad) {
    const int64_t rows = a.transB ? a.N : a.K, cols = a.transB ? a.K : a.N;
    if (a.K > 0) {
      if (!a.C || a.ldc < cols) return GEMM_ERR_INVALID_VALUE;
      // the matrices follow each other, or lie side by side in rows of ldc elements
      const bool apart = (__int128)a.stride_c >= (__int128)(rows - 1) * a.ldc + cols;
      const bool beside = a.stride_c >= cols && (__int128)(a.groups - 1) * a.stride_c + cols <= a.ldc;
      if (a.groups > 1 && !apart && !beside) return GEMM_ERR_INVALID_VALUE;
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

constexpr int64_t kMaxRowBytes = int64_t(1) << 23;  // the kernels' 32-bit lane offsets span up to 256 rows
// (A leading dimension may be any number where there is one row: no product with its size.)
bool short_rows(int64_t ld, int size) { return ld <= kMaxRowBytes / size; }
// ld elements are whole 16-byte chunks.
bool whole_chunks(int64_t ld, int size) { return ld % (16 / size) == 0; }

// The tiled kernels read 16-byte chunks of both operands and store runs of C.
bool tiles_fit(const GArgs& a) {
  const int in = a.i8 ? 1 : es(a.at);
  auto rows_ok = [&](const void* p, int64_t ld) {
    return aligned(p, 16) && whole_chunks(ld, in) && short_rows(ld, in);
  };
  const bool reads = a.wgrad ? a.M > 0 : a.K > 0;
  if (reads && (!rows_ok(a.A, a.lda) || !rows_ok(a.B, a.ldb) || !whole_chunks(a.stride_b, in))) return false;
  return aligned(a.C, 16) && a.ldc % 4 == 0 && a.stride_c % 4 == 0;
}
// The streaming kernel takes any alignment; stored K x N, four columns at a time.  Its smallest
// workgroups have 16 rows of 32 (N x K) or 64 columns.
bool stream_fits(const GArgs& a) {
  const int in = a.i8 ? 1 : es(a.at);
  return !a.wgrad && (a.transB || a.N >= 4) && short_rows(a.lda, in) && short_rows(a.ldb, in) &&
         countable(tgemm::max_row_tiles(a.M, a.groups, 16), a.N, a.transB ? 32 : 64);
}

// Groups that can hold rows, and the rows of one on average.
int64_t live_groups(const GArgs& a) { return a.groups < a.M ? a.groups : a.M; }

// Row tiles of height bm to expect: every group's last one is half empty on average (a single
// group's number is known).
int64_t expected_tiles(const GArgs& a, int64_t bm, int64_t bn) {
  const int64_t rows = a.groups == 1 ? (a.M + bm - 1) / bm : (a.M + live_groups(a) * (bm / 2) + bm - 1) / bm;
  return rows * ((a.N + bn - 1) / bn);
}

gemm_grouped_kernel_t pick(const GArgs& a, int cus) {
  const int64_t rows = (a.M + live_groups(a) - 1) / (live_groups(a) > 0 ? live_groups(a) : 1);
  if (a.wgrad) {
    // Narrow gradients of few rows are all epilogue: the copies through registers take the least LDS,
    // so that four workgroups share a compute unit (19 groups of 2944 x 64 bf16 from 9 rows 8 us against
    // 13 on large tiles, 85 of 6168 x 128 fp16 from 14986 rows 157 against 187).
    if (!tiles_fit(a) || ((a.N < 192 || a.K < 192) && rows <= 256)) return GEMM_GROUPED_ANY;
    auto tiles = [&](int64_t bm, int64_t bn) { return (a.N + bm - 1) / bm * ((a.K + bn - 1) / bn) * a.groups; };
    // large tiles from 5/8 of a round on: 5 groups of 1744 x 1424 (210 tiles) 16 us against 23 on
    // 128 x 128 ones, 4 of 2608 x 704 (132) 18 against 16
    if (8 * tiles(256, 256) >= 5 * cus) return GEMM_GROUPED_MFMA_256;
    if (tiles(128, 128) >= cus / 2) return GEMM_GROUPED_MFMA_128;
    return GEMM_GROUPED_MFMA_64;
  }
  // Few rows a group: what counts is the weights' bytes, and the streaming kernel reads them at the
  // rate of the memory, but the rows once for every 32 or 64 columns.  How far that carries depends
  // on whether 128 x 128 tiles, one row of them to a group, would fill the compute units (32 groups of
  // 2048 x 2048 bf16, B as N x K: 6 rows a group 56 us against 65 on tiles, 16 rows 69 against 65, 32
  // rows 112 against 72; as K x N 2 rows 46 against 48, 6 rows 54 against 51), or not (one group,
  // N 8192, K 4096: 32 rows 18 against 21 and 48 rows 23 against 21; as K x N 64 rows 19 against 23), and on
  // there being tiles for the alignment (without: 16 rows 69 against 71, 32 rows 112 against 105).
  const bool fits = tiles_fit(a), kn = a.transB == 0, many = live_groups(a) * ((a.N + 127) / 128) >= cus;
  const int64_t most = fits ? (many ? (kn ? 4 : 8) : (kn ? 64 : 32)) : (kn ? 64 : many ? 24 : 48);
  // Few 64 x 64 tiles stream too: more waves share out K (1584 rows over 2 groups, N 80, K 5832, bf16
  // 23 us against 30 on 64 x 64 tiles, 236 x 688 x 1824 fp16 9 against 13; 545 rows over 6 groups, N
  // 984, K 1432, whose tiles fill most compute units, 19 against 13).
  if (stream_fits(a) && (rows <= most || 4 * expected_tiles(a, 64, 64) <= cus)) return GEMM_GROUPED_STREAM;
  // So is a K of at most one and a half K tiles (2439 x 2480 x 160 in 8 bits 15 us against 18 on large
  // tiles, 207 rows over 16 groups, N 6368, K 96, 13 against 22; 10313 x 2368 x 208 over 7 groups 40
  // against 30).
  if (!fits || a.K * (a.i8 ? 1 : 2) <= 192) return GEMM_GROUPED_ANY;
  // Large tiles, mixed with small ones, from half a round on (1710 x 6576 x 5296 in 8 bits over 3
  // groups, 234 of them, 76 us against 100 on 128 x 128 tiles; 120 of them 77 against 79, 66 22 against 21).
  if (2 * expected_tiles(a, 256, 256) >= cus) return GEMM_GROUPED_MFMA_256;
  if (16 * expected_tiles(a, 128, 128) >= 9 * cus) return GEMM_GROUPED_MFMA_128;
  return GEMM_GROUPED_MFMA_64;
}

int tile_of(const GArgs& a, gemm_grouped_kernel_t k, int cus) {  // GroupedTile
  // one 64 x 64 tile a compute unit
  const int64_t tiles = a.wgrad ? (a.N + 63) / 64 * ((a.K + 63) / 64) * a.groups : expected_tiles(a, 64, 64);
  const bool few = tiles <= cus;
  switch (k) {
    case GEMM_GROUPED_ANY: return few ? 5 : 0;
    case GEMM_GROUPED_MFMA_64: return few ? 4 : 1;
    case GEMM_GROUPED_MFMA_128: return 2;
    case GEMM_GROUPED_MFMA_256: return 3;
    default: return 0;
  }
}

// The kernel of a call, or an error: kernels asked for by name have to fit.
gemm_status_t choose(const GArgs& a, int cus, gemm_grouped_kernel_t& k) {
  switch (k) {
    case GEMM_GROUPED_AUTO: k = pick(a, cus); return GEMM_OK;
    case GEMM_GROUPED_ANY: return GEMM_OK;
    case GEMM_GROUPED_STREAM: return stream_fits(a) ? GEMM_OK : GEMM_ERR_UNSUPPORTED;
    case GEMM_GROUPED_MFMA_64:
    case GEMM_GROUPED_MFMA_128:
    case GEMM_GROUPED_MFMA_256: return tiles_fit(a) ? GEMM_OK : GEMM_ERR_UNSUPPORTED;
    default: return GEMM_ERR_INVALID_VALUE;
  }
}

gemm_status_t run_rows(gemm_handle_t h, gemm_grouped_kernel_t kernel, void* stream, const GArgs& a, float alpha,
                       float beta, void* C) {
  if (!valid(h)) return GEMM_ERR_INVALID_HANDLE;
  gemm_status_t st = check(a);
  if (st != GEMM_OK) return st;
  if (a.M == 0 || a.N == 0 || a.groups == 0) return GEMM_OK;
  if ((st = choose(a, h->cu_count, kernel)) != GEMM_OK) return st;
  tgemm::GemmParams p = params(a, alpha, beta, C);
  p.bias = (a.epi & GEMM_EPI_BIAS) ? a.bias : nullptr;
  p.ra = a.sa;
  p.rb = a.sb;
  const tgemm::GroupArgs ga{a.offsets, (int)a.groups, a.stride_b, 0, 0};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool kn = a.transB == 0;
  tgemm::DeviceGuard g(h->device);
  if (kernel == GEMM_GROUPED_STREAM) {
    // rows of a workgroup: what a group has on average, less while there are compute units to spare
    // (the weights are then read once more, from the L2, but by more waves)
    const int64_t avg = (a.M + live_groups(a) - 1) / live_groups(a);
    int rows = avg <= (a.groups == 1 ? 16 : 10) ? 16 : avg <= (a.groups == 1 ? 32 : 24) ? 32 : 64;
    while (rows > 16 && 4 * expected_tiles(a, rows, kn ? 64 : 32) <= 3 * h->cu_count) rows /= 2;
    const bool one = expected_tiles(a, rows, kn ? 64 : 32) <= h->cu_count;  // workgroup a compute unit
    const int waves = rows == 64 && kn ? 4 : rows == 16 && one ? 16 : 8;  // (at most 64 KB of LDS)
    return status(a.i8              ? tgemm::launch_stream_i8(p, ga, a.ct, kn, rows, waves, s)
                  : a.at == GEMM_F16 ? tgemm::launch_stream_f16(p, ga, a.ct, kn, rows, waves, s)
                                     : tgemm::launch_stream_bf16(p, ga, a.ct, kn, rows, waves, s));
  }
  const int tile = tile_of(a, kernel, h->cu_count);
  if (!a.i8) return status(a.at == GEMM_F16 ? tgemm::launch_grouped_f16(p, ga, kn, tile, h->cu_count, s) : tgemm::launch_grouped_bf16(p, ga, kn, tile, h->cu_count, s));
  return status(a.ct == GEMM_F32   ? tgemm::launch_grouped_i8_f32(p, ga, kn, tile, h->cu_count, s)
                : a.ct == GEMM_F16 ? tgemm::launch_grouped_i8_f16(p, ga, kn, tile, h->cu_count, s)
                                   : tgemm::launch_grouped_i8_bf16(p, ga, kn, tile, h->cu_count, s));
}

gemm_status_t run_wgrad(gemm_handle_t h, gemm_grouped_kernel_t kernel, void* stream, const GArgs& a, float alpha,
                        float beta, void* C, float* dbias) {
  if (!valid(h)) return GEMM_ERR_INVALID_HANDLE;
  gemm_status_t st = check(a);
  if (st != GEMM_OK) return st;
  if (a.N == 0 || a.groups == 0 || (a.K == 0 && !dbias)) return GEMM_OK;
  if (kernel == GEMM_GROUPED_STREAM) return GEMM_ERR_UNSUPPORTED;
  if ((st = choose(a, h->cu_count, kernel)) != GEMM_OK) return st;
  const tgemm::GroupArgs ga{a.offsets, (int)a.groups, 0, a.stride_c, 0};
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
  const tgemm::BiasGrad b{a.B, a.ldb, (int)a.N, 0, 0, dbias};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  tgemm::DeviceGuard g(h->device);
  return status(a.at == GEMM_F16 ? tgemm::launch_grouped_wgrad_f16(p, ga, b, a.ct, tile_of(a, kernel, h->cu_count), s)
                                 : tgemm::launch_grouped_wgrad_bf16(p, ga, b, a.ct, tile_of(a, kernel, h->cu_count), s));
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
