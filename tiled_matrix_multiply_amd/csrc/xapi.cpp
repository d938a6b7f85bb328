// Host side of the entry points declared in include/gemm_experts.h: argument validation, kernel choice
// and launches.  Nothing is allocated per call, and places and offsets are never read here.
#include "gemm_experts.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "checks.hpp"
#include "experts.hpp"
#include "grouped.hpp"
#include "handle.hpp"

namespace tgemm {
hipError_t launch_route(const RouteArgs&, hipStream_t);
hipError_t launch_route_grad(const RouteGradArgs&, hipStream_t);
hipError_t launch_dispatch_rows(const RowArgs&, int type, hipStream_t);
hipError_t launch_combine_rows(const RowArgs&, int type, hipStream_t);
hipError_t launch_combine_rows_grad(const RowGradArgs&, int type, hipStream_t);
hipError_t launch_quantize_mx(const QuantizeMxArgs&, int x_type, hipStream_t);
hipError_t launch_stream_mx(const GemmParams&, const GroupArgs&, int c_type, int rows, int columns, hipStream_t);
// grouped_mfma.hpp's tiles (its GroupedTile numbers)
hipError_t launch_grouped_mx_f16(const GemmParams&, const GroupArgs&, int tile, int cus, hipStream_t);
hipError_t launch_grouped_mx_bf16(const GemmParams&, const GroupArgs&, int tile, int cus, hipStream_t);
hipError_t launch_grouped_mx_f32(const GemmParams&, const GroupArgs&, int tile, int cus, hipStream_t);
}  // namespace tgemm

namespace {

using namespace tgemm::checks;

constexpr int64_t kMaxGroups = 65535;
constexpr int64_t kMaxTokens = int64_t(1) << 29;  // of the router: 4 threads a token at least, counted in 32 bits
constexpr int64_t kMaxExperts = 1024, kMaxTop = 32, kMaxRuns = 64;

// Whether a result overlaps an operand or another result.
bool aliased(std::initializer_list<Range> out, std::initializer_list<Range> in) {
  for (const Range* a = out.begin(); a != out.end(); ++a) {
    for (const Range& b : in)
      if (overlaps(*a, b)) return true;
    for (const Range* b = a + 1; b != out.end(); ++b)
      if (overlaps(*a, *b)) return true;
  }
  return false;
}

// Pairs of tokens and experts are counted in 31 bits.
bool pairs_fit(int64_t tokens, int64_t top) { return (__int128)tokens * top <= kMaxDim; }

gemm_status_t check_sizes(int64_t T, int64_t E, int64_t top, gemm_dtype_t xt, int score, int renorm) {
  if (T < 0 || E < 1 || top < 1 || top > E) return GEMM_ERR_INVALID_VALUE;
  if (score != GEMM_SCORE_SOFTMAX && score != GEMM_SCORE_SIGMOID) return GEMM_ERR_INVALID_VALUE;
  if (renorm != 0 && renorm != 1) return GEMM_ERR_INVALID_VALUE;
  if (!es(xt) || T > kMaxTokens || E > kMaxExperts || top > kMaxTop || !pairs_fit(T, top)) return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

int64_t route_bytes(int64_t T, int64_t E) {
  return T <= tgemm::route_alone(E) ? 0 : tgemm::route_blocks(T, E) * tgemm::route_row_bytes(E);
}

gemm_status_t check_route(int64_t T, int64_t E, int64_t top, const void* x, int64_t ldl, gemm_dtype_t xt, int score,
                          const float* bias, int64_t groups, int64_t top_groups, int group_top, int renorm,
                          const int32_t* expert, const float* weight, const int32_t* place, const int64_t* offsets,
                          const void* ws, int64_t ws_bytes) {
  const gemm_status_t st = check_sizes(T, E, top, xt, score, renorm);
  if (st != GEMM_OK) return st;
  if (groups < 1 || E % groups != 0 || top_groups < 1 || top_groups > groups) return GEMM_ERR_INVALID_VALUE;
  if (group_top != 1 && group_top != 2) return GEMM_ERR_INVALID_VALUE;
  if (top > top_groups * (E / groups)) return GEMM_ERR_INVALID_VALUE;
  if (groups > kMaxRuns) return GEMM_ERR_UNSUPPORTED;
  if (!offsets || !aligned(offsets, 8) || ws_bytes < 0) return GEMM_ERR_INVALID_VALUE;
  const int64_t need = route_bytes(T, E);
  if (need > 0 && (!ws || ws_bytes < need || !aligned(ws, 16))) return GEMM_ERR_INVALID_VALUE;
  if (T > 0 && (!x || ldl < E || !expert || !weight || !place)) return GEMM_ERR_INVALID_VALUE;
  const Range rx = range(x, T, E, ldl, es(xt)), rb = range(bias, 1, E, 0, 4), ro = range(offsets, 1, E + 1, 0, 8);
  const Range re = range(expert, 1, T * top, 0, 4), rw = range(weight, 1, T * top, 0, 4);
  const Range rp = range(place, 1, T * top, 0, 4), rs = range(ws, 1, need, 0, 1);
  return aliased({re, rw, rp, ro, rs}, {rx, rb}) ? GEMM_ERR_ALIAS : GEMM_OK;
}

gemm_status_t check_route_grad(int64_t T, int64_t E, int64_t top, const void* x, int64_t ldl, gemm_dtype_t xt, int score,
                               int renorm, const int32_t* expert, const float* dw, const void* dx, int64_t ldd) {
  const gemm_status_t st = check_sizes(T, E, top, xt, score, renorm);
  if (st != GEMM_OK || T == 0) return st;
  if (!x || ldl < E || !expert || !dw || !dx || ldd < E) return GEMM_ERR_INVALID_VALUE;
  const Range rx = range(x, T, E, ldl, es(xt)), re = range(expert, 1, T * top, 0, 4), rw = range(dw, 1, T * top, 0, 4);
  return aliased({range(dx, T, E, ldd, es(xt))}, {rx, re, rw}) ? GEMM_ERR_ALIAS : GEMM_OK;
}

// What the moves of rows have in common.
gemm_status_t check_move(int64_t T, int64_t top, int64_t K, gemm_dtype_t type, int64_t R) {
  if (T < 0 || top < 1 || K < 0 || R < 0) return GEMM_ERR_INVALID_VALUE;
  if (!es(type) || T > kMaxDim || K > kMaxDim || R > kMaxDim || !pairs_fit(T, top)) return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

gemm_status_t check_dispatch(int64_t T, int64_t top, int64_t K, const void* X, int64_t ldx, gemm_dtype_t type,
                             const int32_t* place, int64_t R, const void* A, int64_t lda) {
  const gemm_status_t st = check_move(T, top, K, type, R);
  if (st != GEMM_OK || T == 0 || K == 0 || R == 0) return st;
  if (!X || ldx < K || !place || !A || lda < K) return GEMM_ERR_INVALID_VALUE;
  const int e = es(type);
  const Range rx = range(X, T, K, ldx, e), rp = range(place, 1, T * top, 0, 4), ra = range(A, R, K, lda, e);
  return aliased({ra}, {rx, rp}) ? GEMM_ERR_ALIAS : GEMM_OK;
}

gemm_status_t check_combine(int64_t T, int64_t top, int64_t K, const void* Y, int64_t ldy, gemm_dtype_t type,
                            const int32_t* place, int64_t R, const float* weight, const void* C, int64_t ldc) {
  const gemm_status_t st = check_move(T, top, K, type, R);
  if (st != GEMM_OK || T == 0 || K == 0) return st;
  if (!place || !C || ldc < K || (R > 0 && (!Y || ldy < K))) return GEMM_ERR_INVALID_VALUE;
  const int e = es(type);
  const Range ry = range(Y, R, K, ldy, e), rp = range(place, 1, T * top, 0, 4), rw = range(weight, 1, T * top, 0, 4);
  return aliased({range(C, T, K, ldc, e)}, {ry, rp, rw}) ? GEMM_ERR_ALIAS : GEMM_OK;
}

gemm_status_t check_combine_grad(int64_t T, int64_t top, int64_t K, const void* D, int64_t ldd, const void* Y,
                                 int64_t ldy, gemm_dtype_t type, const int32_t* place, int64_t R, const float* weight,
                                 const void* dY, int64_t lddy, const float* dw) {
  const gemm_status_t st = check_move(T, top, K, type, R);
  if (st != GEMM_OK || T == 0) return st;
  if (!place || !weight || !dw) return GEMM_ERR_INVALID_VALUE;
  if (K > 0 && (!D || ldd < K || (R > 0 && (!Y || ldy < K || !dY || lddy < K)))) return GEMM_ERR_INVALID_VALUE;
  const int e = es(type);
  const Range rd = range(D, T, K, ldd, e), ry = range(Y, R, K, ldy, e), ro = range(dY, R, K, lddy, e);
  const Range rp = range(place, 1, T * top, 0, 4), rw = range(weight, 1, T * top, 0, 4), rg = range(dw, 1, T * top, 0, 4);
  return aliased({ro, rg}, {rd, ry, rp, rw}) ? GEMM_ERR_ALIAS : GEMM_OK;
}

gemm_status_t check_quantize(int64_t M, int64_t K, const void* X, int64_t ldx, gemm_dtype_t xt, int64_t top,
                             const int32_t* place, int64_t R, const void* Q, int64_t ldq, gemm_dtype_t qt,
                             const uint8_t* S, int64_t lds) {
  const gemm_status_t st = check_move(M, top, K, xt, R);
  if (st != GEMM_OK) return st;
  if (qt != GEMM_E2M1) return GEMM_ERR_UNSUPPORTED;
  if (K % 32 != 0 || (!place && (top != 1 || R != M))) return GEMM_ERR_INVALID_VALUE;
  if (M == 0 || K == 0 || R == 0) return GEMM_OK;
  if (!X || ldx < K || !Q || ldq < K || ldq % 2 != 0 || !S || lds < K / 32) return GEMM_ERR_INVALID_VALUE;
  const Range rx = range(X, M, K, ldx, es(xt)), rp = range(place, 1, M * top, 0, 4);
  const Range rq = range(Q, R, K / 2, ldq / 2, 1), rs = range(S, R, K / 32, lds, 1);
  return aliased({rq, rs}, {rx, rp}) ? GEMM_ERR_ALIAS : GEMM_OK;
}

struct MxArgs {
  int64_t groups;
  const int64_t* offsets;
  int64_t M, N, K;
  const void* A;
  int64_t lda;
  const uint8_t* sa;
  int64_t ldsa;
  const void* B;
  int64_t ldb, stride_b;
  const uint8_t* sb;
  int64_t ldsb, stride_sb;
  const void* C;
  int64_t ldc;
  gemm_dtype_t type, ct;
  uint32_t epi;
  const float* bias;
};

// Workgroups must be countable in 31 bits, with the worst case's row tiles and a last round of 8.
bool countable(const MxArgs& a, int64_t bm, int64_t bn) {
  return (__int128)tgemm::max_row_tiles(a.M, a.groups, bm) * ((a.N + bn - 1) / bn) <= kMaxDim - 16;
}

gemm_status_t check(const MxArgs& a) {
  if (a.M < 0 || a.N < 0 || a.K < 0 || a.groups < 0) return GEMM_ERR_INVALID_VALUE;
  if (a.epi & ~(GEMM_EPI_BIAS | GEMM_EPI_GELU)) return GEMM_ERR_INVALID_VALUE;
  if (a.type != GEMM_E2M1 || !es(a.ct)) return GEMM_ERR_UNSUPPORTED;
  if (a.M > kMaxDim || a.N > kMaxDim || a.K > kMaxDim || a.groups > kMaxGroups) return GEMM_ERR_UNSUPPORTED;
  if (a.K % 32 != 0) return GEMM_ERR_INVALID_VALUE;
  if (a.M == 0 || a.N == 0 || a.groups == 0) return GEMM_OK;  // nothing to compute
  if (!countable(a, 64, 32)) return GEMM_ERR_UNSUPPORTED;
  if ((!a.offsets && a.groups != 1) || !aligned(a.offsets, 8)) return GEMM_ERR_INVALID_VALUE;
  if (!a.C || a.ldc < a.N || a.stride_b < 0 || a.stride_sb < 0) return GEMM_ERR_INVALID_VALUE;
  if ((a.epi & GEMM_EPI_BIAS) && !a.bias) return GEMM_ERR_INVALID_VALUE;
  const Range rc = range(a.C, a.M, a.N, a.ldc, es(a.ct));
  if (a.K > 0) {
    if (!a.A || !a.B || !a.sa || !a.sb || a.lda < a.K || a.ldb < a.K) return GEMM_ERR_INVALID_VALUE;
    if (a.lda % 2 != 0 || a.ldb % 2 != 0 || a.stride_b % 2 != 0) return GEMM_ERR_INVALID_VALUE;
    if (a.ldsa < a.K / 32 || a.ldsb < a.K / 32) return GEMM_ERR_INVALID_VALUE;
    if (aliased({rc}, {range(a.A, a.M, a.K / 2, a.lda / 2, 1), range(a.sa, a.M, a.K / 32, a.ldsa, 1),
                       range(a.B, a.N, a.K / 2, a.ldb / 2, 1, a.groups, a.stride_b / 2),
                       range(a.sb, a.N, a.K / 32, a.ldsb, 1, a.groups, a.stride_sb)}))
      return GEMM_ERR_ALIAS;
  }
  if (overlaps(rc, range(a.offsets, 1, a.groups + 1, 0, 8))) return GEMM_ERR_ALIAS;
  if ((a.epi & GEMM_EPI_BIAS) && overlaps(rc, range(a.bias, 1, a.groups * a.N, 0, 4))) return GEMM_ERR_ALIAS;
  return GEMM_OK;
}

// A leading dimension counts where there is a second row.
int64_t step(int64_t ld, int64_t rows, int64_t least) { return rows > 1 ? ld : least; }

bool stream_fits(const MxArgs& a) {
  const int64_t most = kMaxRowBytes;
  return step(a.lda, a.M, a.K) <= 2 * most && step(a.ldb, a.N, a.K) <= 2 * most && step(a.ldsa, a.M, 0) <= most &&
         step(a.ldsb, a.N, 0) <= most && countable(a, 64, 32);
}

// The tiled kernels copy 16-byte chunks of the operands and their scales and store runs of C.
bool tiles_fit(const MxArgs& a) {
  if (!aligned(a.C, 16) || a.ldc % 4 != 0) return false;
  if (a.K == 0) return true;
  const int64_t most = kMaxRowBytes;
  auto scales_fit = [](int64_t ld, int64_t rows) { return ld % 16 == 0 && (__int128)ld * rows < ((__int128)1 << 32); };
  return aligned(a.A, 16) && aligned(a.B, 16) && aligned(a.sa, 16) && aligned(a.sb, 16) && a.lda % 32 == 0 &&
         a.ldb % 32 == 0 && a.stride_b % 32 == 0 && a.lda <= 2 * most && a.ldb <= 2 * most && a.stride_sb % 16 == 0 &&
         scales_fit(a.ldsa, a.M) && scales_fit(a.ldsb, a.N);
}

// Groups that can hold rows, and the row tiles of height bm to expect: every group's last one is half
// empty on average (a single group's number is known).
int64_t live_groups(const MxArgs& a) { return a.groups < a.M ? a.groups : a.M; }
int64_t expected_tiles(const MxArgs& a, int64_t bm, int64_t bn) {
  const int64_t rows = a.groups == 1 ? (a.M + bm - 1) / bm : (a.M + live_groups(a) * (bm / 2) + bm - 1) / bm;
  return rows * ((a.N + bn - 1) / bn);
}

// Rows of a group that has any, on average.
int64_t average_rows(const MxArgs& a) { return (a.M + live_groups(a) - 1) / live_groups(a); }

// Rows and columns of a streaming workgroup (times: one MI355X, constant operands, 256 compute units).
struct StreamTile {
  int rows, columns, cost;
};
StreamTile stream_tile(const MxArgs& a, int cus) {
  // Up to 8 rows of one group: the weights' way from memory counts, and more workgroups even out the last
  // round (1 x 4096 x 4096 4.0 us against 5.2 with 32 columns, 1 x 20480 x 7168 14.3 against 15.7, 1 x 16384 x
  // 7168, two for each unit exactly, 12.1 against 11.4).
  if (a.groups == 1 && a.M <= 8 && countable(a, 16, 16)) return {16, 16, 0};
  if (a.groups == 1) {
    // More rows of one group: the caches' rate counts, and a compute unit with two workgroups takes almost
    // twice as long.  A round of each kind (K of 8192: 7.1, 9.4, 12 and 17.6 us; of 2048: 4.1, 4.4, 5.2 and 7.0)
    // costs about 9, 14, 19 and 30.  37 x 4104 x 4128: 387 of 16 x 32 6.6 us, 258 of 32 x 32 7.2, 129 of 64 x 32
    // 7.4; 37 x 4096 x 4096: 384, 256 and 128 of them 9.4, 7.7 and 9.0.
    const StreamTile kinds[] = {{16, 16, 9}, {16, 32, 14}, {32, 32, 19}, {64, 32, 30}};
    StreamTile best{64, 32, 0x7fffffff};
    for (const StreamTile& t : kinds) {
      const int64_t rounds = (expected_tiles(a, t.rows, t.columns) + cus - 1) / cus;
      if (rounds < 1000 && rounds * t.cost < best.cost && countable(a, t.rows, t.columns))
        best = {t.rows, t.columns, (int)rounds * t.cost};
    }
    return best;
  }
  // Groups: as few rows as leave the compute units at most 1.6 workgroups each, up to twice the average, and
  // half the columns where that is not one each (8 rows in each of 32 groups of 1024 x 4096: 16 x 32 18.8 us, 32 x 32
  // 17.3, 64 x 32 20.3; 4 in each of 4 of 1024 x 4096: 16 x 16 4.7, 16 x 32 5.6).
  const int64_t most = 2 * average_rows(a);
  int rows = 16;
  while (rows < 64 && ((rows < most && 10 * expected_tiles(a, rows, 32) > 16 * cus) || !countable(a, rows, 32))) rows *= 2;
  const bool narrow = rows == 16 && countable(a, 16, 16) && expected_tiles(a, 16, 16) <= cus;
  return {rows, narrow ? 16 : 32, 0};
}

// The kernel of a call (times as above).
gemm_grouped_kernel_t pick(const MxArgs& a, int cus) {
  const int64_t rows = average_rows(a), small = expected_tiles(a, 64, 64);
  if (!tiles_fit(a)) return GEMM_GROUPED_STREAM;
  if (stream_fits(a)) {
    // Streaming needs no barrier and starts at once, but reads half lines, and the rows once for every 16 or
    // 32 columns: it pays where 64 x 64 tiles are few.  One group: always up to 8 rows (1 x 28672 x 8192 24 us
    // against 28); with more, up to three rounds of 16 x 16, two of 16 x 32 or one of 32 x 32 (256 x 1024 x 4096, one
    // of 32 x 32, 7.6 against 10.3; 320 x 1600 x 8192, one of 64 x 32, 17.9 against 17.3; 16 x 28672 x 8192 37
    // against 31).
    // Many: 64 rows over 8 groups of 1024 x 1024 (80) 3.7 against 5.2, 32 over 64 of 1024 x 2048 (272) 8.2 against
    // 9.5, 64 over 32 of 2048 x 2048 (544, 2 rows a group) 13.5 against 14.2, 256 rows 16.2 against 14.2, 128 over
    // 16 of 4096 x 4096 (640) 38 against 30.
    if (a.groups == 1) {
      if (stream_tile(a, cus).cost <= 28) return GEMM_GROUPED_STREAM;
    } else if ((rows <= 32 && 4 * small <= (rows <= 4 ? 10 : 5) * cus) || (rows <= 128 && 4 * small <= cus)) {
      return GEMM_GROUPED_STREAM;
    }
  }
  // Large tiles, mixed with small ones, from 5/8 of a round on, with uneven groups from 3/8 on if they hold
  // large tiles at all (1536 x 8192 x 1024, 192 of them, 13.5 us against 15.1 on 128 x 128 ones, 2048 x 4096 x
  // 4096, 128, 33 against 23; 4096 rows over 8 uneven groups of 2048 x 2048, 128, 18.1 against 22.9 (even groups
  // 22.8 against 15.6), but 4096 over 32 of 2048 x 2048, 128, 30 against 27).
  const int64_t large = a.M * ((a.N + 255) / 256);  // in rows of 256
  if (a.groups == 1 ? 8 * large >= 5 * 256 * cus : rows >= 160 && 8 * large >= 3 * 256 * cus) return GEMM_GROUPED_MFMA_256;
  // 128 x 128 from 13/16 of a round on (1024 x 3456 x 2048, 216 of them, 10.7 us against 11.6 on 64 x 64 ones, 2048 x
  // 1536 x 2048, 192, 10.7 against 10.0), with GELU, which takes longest where one round has a few waves only, from
  // 9/8 (1024 x 4096 x 2048, 256, 15.0 against 13.4, 2048 x 2560 x 2048, 320, 17.9 against 19.7), and with rows
  // that fill them (64 rows a group 23.5 against 19.0, 128 rows 26.8 against 28.7: 32 uneven groups of 2048 x 2048;
  // 32 x 28672 x 4096 17.8 against 14.5).
  const int least = a.epi & GEMM_EPI_GELU ? 18 : 13;
  if (rows >= 96 && 16 * expected_tiles(a, 128, 128) >= least * cus) return GEMM_GROUPED_MFMA_128;
  return GEMM_GROUPED_MFMA_64;
}

gemm_status_t run(gemm_handle_t h, gemm_grouped_kernel_t kernel, void* stream, const MxArgs& a, float alpha, float beta,
                  void* C) {
  if (!valid(h)) return GEMM_ERR_INVALID_HANDLE;
  const gemm_status_t st = check(a);
  if (st != GEMM_OK) return st;
  if (kernel < GEMM_GROUPED_AUTO || kernel > GEMM_GROUPED_STREAM) return GEMM_ERR_INVALID_VALUE;
  if (a.M == 0 || a.N == 0 || a.groups == 0) return GEMM_OK;
  if (kernel == GEMM_GROUPED_AUTO) kernel = pick(a, h->cu_count);
  if (kernel == GEMM_GROUPED_ANY || !(kernel == GEMM_GROUPED_STREAM ? stream_fits(a) : tiles_fit(a)))
    return GEMM_ERR_UNSUPPORTED;
  tgemm::GemmParams p{};
  p.A = a.A;
  p.B = a.B;
  p.C = C;
  p.bias = (a.epi & GEMM_EPI_BIAS) ? a.bias : nullptr;
  p.M = (int)a.M;
  p.N = (int)a.N;
  p.K = (int)(a.K / 2);  // packed rows are bytes to the kernels
  p.lda = step(a.lda, a.M, a.K) / 2;
  p.ldb = step(a.ldb, a.N, a.K) / 2;
  p.ldc = a.ldc;
  p.alpha = alpha;
  p.beta = beta;
  p.epi = a.epi;
  p.sa = a.sa;
  p.sb = a.sb;
  p.ldsa = a.ldsa;
  p.ldsb = a.ldsb;
  p.kblocks = (int)(a.K / 32);
  const tgemm::GroupArgs ga{a.offsets, (int)a.groups, a.stride_b / 2, 0, 0, a.stride_sb};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  tgemm::DeviceGuard g(h->device);
  if (kernel == GEMM_GROUPED_STREAM) {
    const StreamTile t = stream_tile(a, h->cu_count);
    p.ldsa = step(a.ldsa, a.M, 0);
    p.ldsb = step(a.ldsb, a.N, 0);
    return status(tgemm::launch_stream_mx(p, ga, a.ct, t.rows, t.columns, s));
  }
  const bool deep = a.K >= 4096 && expected_tiles(a, 64, 64) <= 2 * h->cu_count;  // three stages (GroupedMxCfg)
  const int tile = kernel == GEMM_GROUPED_MFMA_64 ? (deep ? 4 : 1) : kernel == GEMM_GROUPED_MFMA_128 ? 2 : 3;
  return status(a.ct == GEMM_F32   ? tgemm::launch_grouped_mx_f32(p, ga, tile, h->cu_count, s)
                : a.ct == GEMM_F16 ? tgemm::launch_grouped_mx_f16(p, ga, tile, h->cu_count, s)
                                   : tgemm::launch_grouped_mx_bf16(p, ga, tile, h->cu_count, s));
}

}  // namespace

extern "C" {

int64_t gemm_route_workspace_bytes(int64_t tokens, int64_t experts) {
  if (tokens < 0 || experts < 1) return GEMM_ERR_INVALID_VALUE;
  if (tokens > kMaxTokens || experts > kMaxExperts) return GEMM_ERR_UNSUPPORTED;
  return route_bytes(tokens, experts);
}

gemm_status_t gemm_check_args_route(int64_t tokens, int64_t experts, int64_t top, const void* logits, int64_t ldl,
                                    gemm_dtype_t x_type, gemm_score_t score, const float* bias, int64_t groups,
                                    int64_t top_groups, int group_top, int renorm, const int32_t* expert,
                                    const float* weight, const int32_t* place, const int64_t* offsets,
                                    const void* workspace, int64_t workspace_bytes) {
  return check_route(tokens, experts, top, logits, ldl, x_type, score, bias, groups, top_groups, group_top, renorm, expert,
                     weight, place, offsets, workspace, workspace_bytes);
}

gemm_status_t gemm_route(gemm_handle_t h, void* stream, int64_t tokens, int64_t experts, int64_t top, const void* logits,
                         int64_t ldl, gemm_dtype_t x_type, gemm_score_t score, const float* bias, int64_t groups,
                         int64_t top_groups, int group_top, int renorm, float scale, int32_t* expert, float* weight,
                         int32_t* place, int64_t* offsets, void* workspace, int64_t workspace_bytes) {
  if (!valid(h)) return GEMM_ERR_INVALID_HANDLE;
  const gemm_status_t st = check_route(tokens, experts, top, logits, ldl, x_type, score, bias, groups, top_groups,
                                       group_top, renorm, expert, weight, place, offsets, workspace, workspace_bytes);
  if (st != GEMM_OK) return st;
  const tgemm::RouteArgs p{logits, ldl, (int)tokens, (int)experts, (int)top, (int)x_type, (int)score, bias, (int)groups,
                           (int)top_groups, group_top, renorm, scale, expert, weight, place, offsets,
                           tokens <= tgemm::route_alone(experts) ? nullptr : static_cast<uint8_t*>(workspace), 0, 0, 0};
  tgemm::DeviceGuard g(h->device);
  return status(tgemm::launch_route(p, static_cast<hipStream_t>(stream)));
}

gemm_status_t gemm_check_args_route_grad(int64_t tokens, int64_t experts, int64_t top, const void* logits, int64_t ldl,
                                         gemm_dtype_t x_type, gemm_score_t score, int renorm, const int32_t* expert,
                                         const float* dweight, const void* dlogits, int64_t ldd) {
  return check_route_grad(tokens, experts, top, logits, ldl, x_type, score, renorm, expert, dweight, dlogits, ldd);
}

gemm_status_t gemm_route_grad(gemm_handle_t h, void* stream, int64_t tokens, int64_t experts, int64_t top,
                              const void* logits, int64_t ldl, gemm_dtype_t x_type, gemm_score_t score, int renorm,
                              float scale, const int32_t* expert, const float* dweight, void* dlogits, int64_t ldd) {
  if (!valid(h)) return GEMM_ERR_INVALID_HANDLE;
  const gemm_status_t st =
      check_route_grad(tokens, experts, top, logits, ldl, x_type, score, renorm, expert, dweight, dlogits, ldd);
  if (st != GEMM_OK || tokens == 0) return st;
  const tgemm::RouteGradArgs p{logits, ldl, (int)tokens, (int)experts, (int)top, (int)x_type, (int)score, renorm, scale,
                               expert, dweight, dlogits, ldd};
  tgemm::DeviceGuard g(h->device);
  return status(tgemm::launch_route_grad(p, static_cast<hipStream_t>(stream)));
}

gemm_status_t gemm_check_args_dispatch_rows(int64_t tokens, int64_t top, int64_t K, const void* X, int64_t ldx,
                                            gemm_dtype_t type, const int32_t* place, int64_t rows, const void* A,
                                            int64_t lda) {
  return check_dispatch(tokens, top, K, X, ldx, type, place, rows, A, lda);
}

gemm_status_t gemm_dispatch_rows(gemm_handle_t h, void* stream, int64_t tokens, int64_t top, int64_t K, const void* X,
                                 int64_t ldx, gemm_dtype_t type, const int32_t* place, int64_t rows, void* A,
                                 int64_t lda) {
  if (!valid(h)) return GEMM_ERR_INVALID_HANDLE;
  const gemm_status_t st = check_dispatch(tokens, top, K, X, ldx, type, place, rows, A, lda);
  if (st != GEMM_OK || tokens == 0 || K == 0 || rows == 0) return st;
  const tgemm::RowArgs p{X, ldx, (int)tokens, (int)top, (int)K, (int)rows, place, nullptr, 0.0f, A, lda};
  tgemm::DeviceGuard g(h->device);
  return status(tgemm::launch_dispatch_rows(p, type, static_cast<hipStream_t>(stream)));
}

gemm_status_t gemm_check_args_combine_rows(int64_t tokens, int64_t top, int64_t K, const void* Y, int64_t ldy,
                                           gemm_dtype_t type, const int32_t* place, int64_t rows, const float* weight,
                                           const void* C, int64_t ldc) {
  return check_combine(tokens, top, K, Y, ldy, type, place, rows, weight, C, ldc);
}

gemm_status_t gemm_combine_rows(gemm_handle_t h, void* stream, int64_t tokens, int64_t top, int64_t K, const void* Y,
                                int64_t ldy, gemm_dtype_t type, const int32_t* place, int64_t rows, const float* weight,
                                float beta, void* C, int64_t ldc) {
  if (!valid(h)) return GEMM_ERR_INVALID_HANDLE;
  const gemm_status_t st = check_combine(tokens, top, K, Y, ldy, type, place, rows, weight, C, ldc);
  if (st != GEMM_OK || tokens == 0 || K == 0) return st;
  const tgemm::RowArgs p{Y, ldy, (int)tokens, (int)top, (int)K, (int)rows, place, weight, beta, C, ldc};
  tgemm::DeviceGuard g(h->device);
  return status(tgemm::launch_combine_rows(p, type, static_cast<hipStream_t>(stream)));
}

gemm_status_t gemm_check_args_combine_rows_grad(int64_t tokens, int64_t top, int64_t K, const void* D, int64_t ldd,
                                                const void* Y, int64_t ldy, gemm_dtype_t type, const int32_t* place,
                                                int64_t rows, const float* weight, const void* dY, int64_t lddy,
                                                const float* dweight) {
  return check_combine_grad(tokens, top, K, D, ldd, Y, ldy, type, place, rows, weight, dY, lddy, dweight);
}

gemm_status_t gemm_combine_rows_grad(gemm_handle_t h, void* stream, int64_t tokens, int64_t top, int64_t K,
                                     const void* D, int64_t ldd, const void* Y, int64_t ldy, gemm_dtype_t type,
                                     const int32_t* place, int64_t rows, const float* weight, void* dY, int64_t lddy,
                                     float* dweight) {
  if (!valid(h)) return GEMM_ERR_INVALID_HANDLE;
  const gemm_status_t st = check_combine_grad(tokens, top, K, D, ldd, Y, ldy, type, place, rows, weight, dY, lddy, dweight);
  if (st != GEMM_OK || tokens == 0) return st;
  const tgemm::RowGradArgs p{D, ldd, Y, ldy, (int)tokens, (int)top, (int)K, (int)rows, place, weight, dY, lddy, dweight};
  tgemm::DeviceGuard g(h->device);
  return status(tgemm::launch_combine_rows_grad(p, type, static_cast<hipStream_t>(stream)));
}

gemm_status_t gemm_check_args_quantize_mx(int64_t M, int64_t K, const void* X, int64_t ldx, gemm_dtype_t x_type,
                                          int64_t top, const int32_t* place, int64_t rows, const void* Q, int64_t ldq,
                                          gemm_dtype_t q_type, const uint8_t* S, int64_t lds) {
  return check_quantize(M, K, X, ldx, x_type, top, place, rows, Q, ldq, q_type, S, lds);
}

gemm_status_t gemm_quantize_mx(gemm_handle_t h, void* stream, int64_t M, int64_t K, const void* X, int64_t ldx,
                               gemm_dtype_t x_type, int64_t top, const int32_t* place, int64_t rows, void* Q, int64_t ldq,
                               gemm_dtype_t q_type, uint8_t* S, int64_t lds) {
  if (!valid(h)) return GEMM_ERR_INVALID_HANDLE;
  const gemm_status_t st = check_quantize(M, K, X, ldx, x_type, top, place, rows, Q, ldq, q_type, S, lds);
  if (st != GEMM_OK || M == 0 || K == 0 || rows == 0) return st;
  const tgemm::QuantizeMxArgs p{X, ldx, (int)M, (int)K, (int)top, (int)rows, place, static_cast<uint8_t*>(Q), ldq / 2,
                                S, lds};
  tgemm::DeviceGuard g(h->device);
  return status(tgemm::launch_quantize_mx(p, x_type, static_cast<hipStream_t>(stream)));
}

gemm_status_t gemm_check_args_grouped_mx(int64_t groups, const int64_t* offsets, int64_t M, int64_t N, int64_t K,
                                         const void* A, int64_t lda, const uint8_t* sa, int64_t ldsa, const void* B,
                                         int64_t ldb, int64_t stride_b, const uint8_t* sb, int64_t ldsb,
                                         int64_t stride_sb, const void* C, int64_t ldc, gemm_dtype_t type,
                                         gemm_dtype_t c_type, uint32_t epilogue, const float* bias) {
  return check(MxArgs{groups, offsets, M, N, K, A, lda, sa, ldsa, B, ldb, stride_b, sb, ldsb, stride_sb, C, ldc, type,
                      c_type, epilogue, bias});
}

gemm_status_t gemm_run_grouped_mx(gemm_handle_t h, gemm_grouped_kernel_t kernel, void* stream, int64_t groups,
                                  const int64_t* offsets, int64_t M, int64_t N, int64_t K, float alpha, const void* A,
                                  int64_t lda, const uint8_t* sa, int64_t ldsa, const void* B, int64_t ldb,
                                  int64_t stride_b, const uint8_t* sb, int64_t ldsb, int64_t stride_sb, float beta,
                                  void* C, int64_t ldc, gemm_dtype_t type, gemm_dtype_t c_type, uint32_t epilogue,
                                  const float* bias) {
  const MxArgs a{groups, offsets, M, N, K, A, lda, sa, ldsa, B, ldb, stride_b, sb, ldsb, stride_sb, C, ldc, type, c_type,
                 epilogue, bias};
  return run(h, kernel, stream, a, alpha, beta, C);
}

}  // extern "C"
