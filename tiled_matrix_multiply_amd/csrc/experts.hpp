// Arguments of the kernels behind include/gemm_experts.h (gfx950 only).
#pragma once

#include "common.hpp"

namespace tgemm {

struct RouteArgs {
  const void* x;  // logits
  int64_t ldx;
  int T, E, top;
  int x_type, score;  // DType; 0 softmax, 1 sigmoid
  const float* bias;
  int groups, top_groups, group_top;
  int renorm;
  float scale;
  int32_t* expert;
  float* weight;
  int32_t* place;
  int64_t* offsets;
  uint8_t* ws;  // tokens of each expert in each block, route_row_bytes(E) bytes a block; null: one block
  // set by the launcher
  int run_lanes;  // log2 of the lanes that hold a run of experts; -1: runs do not fit the lanes
  int run_size;   // experts of a run
  int per_top;    // i / top is i * per_top >> 16 for i up to 2048 (off by less than i / 65536 < 1 / top)
};

struct RouteGradArgs {
  const void* x;
  int64_t ldx;
  int T, E, top;
  int x_type, score, renorm;
  float scale;
  const int32_t* expert;
  const float* dw;
  void* dx;
  int64_t ldd;
};

// Tokens that one workgroup of the router takes alone, in one launch: as many as it can hold at a time (64 of
// 256 experts would be two rounds: 12.6 us against 10.0 for 65 in two launches; 64 of 512 four: 24.5 against 10.5).
inline int route_alone(int64_t E) { return E <= 128 ? 64 : E <= 256 ? 32 : 16; }
// Tokens of a workgroup, at most 64: a token is a bit of a 64-bit mask there.  Few where there are few tokens, so
// that they have more compute units; more where there are more, for every workgroup of the second kernel reads
// all workgroups' counts.  Past 256 experts a token has a wave of its own (202 tokens of 416 experts: 13.0 us with
// 4, 14.6 with 16; 1000 of 300: 17.1 and 16.5).
inline int route_block_tokens(int64_t T, int64_t E) {
  if (T <= route_alone(E)) return 64;
  if (E > 256 && T <= 512) return T <= 256 ? 4 : 8;
  return T <= 4096 ? 16 : T <= 8192 ? 32 : 64;
}
inline int64_t route_blocks(int64_t T, int64_t E) { return (T + route_block_tokens(T, E) - 1) / route_block_tokens(T, E); }
constexpr __host__ __device__ int64_t route_row_bytes(int64_t E) { return (E + 15) / 16 * 16; }

struct RowArgs {
  const void* X;  // dispatch: tokens; combine: the experts' rows
  int64_t ldx;
  int T, top, K, R;
  const int32_t* place;
  const float* weight;  // null: 1
  float beta;
  void* Y;
  int64_t ldy;
};

struct RowGradArgs {
  const void* D;
  int64_t ldd;
  const void* Y;
  int64_t ldy;
  int T, top, K, R;
  const int32_t* place;
  const float* weight;
  void* dY;
  int64_t lddy;
  float* dw;
};

struct QuantizeMxArgs {
  const void* X;
  int64_t ldx;
  int M, K, top, R;
  const int32_t* place;  // null: row i to row i
  uint8_t* Q;
  int64_t ldq;  // bytes
  uint8_t* S;
  int64_t lds;
};

}  // namespace tgemm
