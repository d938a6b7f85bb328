// Products grouped by expert: what the kernels share (gfx950 only).
//
// The rows of A and C are sorted by group; a device array of groups + 1 offsets says where each
// group's rows start.  Only the kernels read it: the host sizes the grid for the worst case, and
// every workgroup finds its own group from the offsets (one load per lane, two scans across the
// wave), which costs no launch and no trip to the host.
#pragma once

#include "common.hpp"

namespace tgemm {

struct GroupArgs {
  const int64_t* offsets;  // null: one group that owns every row
  int groups;
  int64_t stride_b;        // elements between the groups' B (rows: forward)
  int64_t stride_c;        // elements between the groups' C (weight gradient)
};

// Upper bound of the row tiles of height bm that any offsets can give M rows.
inline int64_t max_row_tiles(int64_t M, int64_t groups, int64_t bm) {
  const int64_t live = groups < M ? groups : M;  // groups with rows
  return (M + live * (bm - 1)) / bm;
}

// 64 consecutive groups, one per lane: group base + lane owns rows [row0, row0 + rows).
// Offsets are clamped to 0 .. M and raised to the largest before them (`carry`), so groups never
// overlap and never leave the matrix whatever the array holds.
struct GroupLane {
  int row0, rows;
};
__device__ __forceinline__ int clamp_offset(int64_t o, int M) {
  return (int)(o < 0 ? 0 : o > M ? (int64_t)M : o);
}
__device__ __forceinline__ GroupLane group_lane(const GroupArgs& ga, int M, int base, int lane,
                                                int& carry) {
  const int g = base + lane;
  int hi = g < ga.groups ? clamp_offset(ga.offsets[g + 1], M) : 0;
  hi = max(hi, carry);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(hi, d);
    if (lane >= d) hi = max(hi, o);
  }
  int lo = __shfl_up(hi, 1);
  if (lane == 0) lo = carry;
  carry = __shfl(hi, 63);
  return GroupLane{lo, hi - lo};
}

// Rows of one group (wave-uniform).
__device__ __forceinline__ GroupLane group_rows(const GroupArgs& ga, int M, int g, int lane) {
  if (!ga.offsets) return GroupLane{0, M};
  int carry = clamp_offset(ga.offsets[0], M);
  GroupLane r{};
  for (int base = 0; base <= g; base += 64) r = group_lane(ga, M, base, lane, carry);
  return GroupLane{__builtin_amdgcn_readlane(r.row0, g & 63), __builtin_amdgcn_readlane(r.rows, g & 63)};
}

// Work item t of the sequence that lists, group after group, ceil(rows / bm) * per_row items.
struct GroupItem {
  int group;  // -1: t is past the last item
  int row0, rows;
  int local;  // index within the group
};
__device__ __forceinline__ int scan_add(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}
__device__ __forceinline__ int group_items(const GroupArgs& ga, int M, int bm, int per_row, int lane) {
  if (!ga.offsets) return (M + bm - 1) / bm * per_row;
  int carry = clamp_offset(ga.offsets[0], M), total = 0;
  for (int base = 0; base < ga.groups; base += 64) {
    const GroupLane r = group_lane(ga, M, base, lane, carry);
    total += __shfl(scan_add((r.rows + bm - 1) / bm, lane), 63);
  }
  return __builtin_amdgcn_readfirstlane(total) * per_row;
}
__device__ __forceinline__ GroupItem group_item(const GroupArgs& ga, int M, int bm, int per_row, int t,
                                                int lane) {
  if (!ga.offsets) return GroupItem{t < (M + bm - 1) / bm * per_row ? 0 : -1, 0, M, t};
  int carry = clamp_offset(ga.offsets[0], M), before = 0;
  for (int base = 0; base < ga.groups; base += 64) {
    const GroupLane r = group_lane(ga, M, base, lane, carry);
    const int own = (r.rows + bm - 1) / bm, end = before + scan_add(own, lane);
    const uint64_t hit = __ballot((int64_t)end * per_row > t);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      return GroupItem{base + l, __builtin_amdgcn_readlane(r.row0, l), __builtin_amdgcn_readlane(r.rows, l),
                       t - __builtin_amdgcn_readlane(end - own, l) * per_row};
    }
    before = __shfl(end, 63);
  }
  return GroupItem{-1, 0, 0, 0};
}

// Moves the arguments of a product on to one group: its rows of A and C (and their scales), its
// B, bias and column scales.
template <int ES, int CES>
__device__ __forceinline__ void enter_group(GemmParams& p, const GroupArgs& ga, int group, int row0, int rows) {
  p.A = reinterpret_cast<const uint8_t*>(p.A) + (int64_t)row0 * p.lda * ES;
  p.B = reinterpret_cast<const uint8_t*>(p.B) + (int64_t)group * ga.stride_b * ES;
  p.C = reinterpret_cast<uint8_t*>(p.C) + (int64_t)row0 * p.ldc * CES;
  p.M = rows;
  if (p.bias) p.bias += (int64_t)group * p.N;
  if (p.ra) p.ra += row0;
  if (p.rb) p.rb += (int64_t)group * p.N;
}

// The same for the weight gradient, whose sum runs over the group's rows: p.K becomes their
// number.
template <int ES, int CES>
__device__ __forceinline__ void enter_group_wgrad(GemmParams& p, const GroupArgs& ga, int group, int row0, int rows) {
  p.A = reinterpret_cast<const uint8_t*>(p.A) + (int64_t)row0 * p.lda * ES;
  p.B = reinterpret_cast<const uint8_t*>(p.B) + (int64_t)row0 * p.ldb * ES;
  p.C = reinterpret_cast<uint8_t*>(p.C) + (int64_t)group * ga.stride_c * CES;
  p.K = rows;
}

}  // namespace tgemm
