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
  int first;               // workgroups before this launch's own (launch_in_slices)
  int64_t stride_sb;       // bytes between the groups' block scales of B (microscaled products)
};

__device__ __forceinline__ int workgroup(const GroupArgs& ga) { return ga.first + (int)blockIdx.x; }

// Upper bound of the row tiles of height bm that any offsets can give M rows.
inline int64_t max_row_tiles(int64_t M, int64_t groups, int64_t bm) {
  const int64_t live = groups < M ? groups : M;  // groups with rows
  return (M + live * (bm - 1)) / bm;
}

// Scans across the wave, lane by lane upwards (six vector instructions each, no LDS): the running
// maximum and the running sum of non-negative values.
template <class F>
__device__ __forceinline__ int scan_up(int v, F f) {
  v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));  // row_shr 1, 2, 4, 8
  v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));  // row_bcast 15
  v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));  // row_bcast 31
  return v;
}
__device__ __forceinline__ int scan_max(int v) { return scan_up(v, [](int a, int b) { return max(a, b); }); }
__device__ __forceinline__ int scan_add(int v) { return scan_up(v, [](int a, int b) { return a + b; }); }

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
  hi = scan_max(max(hi, carry));
  const int lo = __builtin_amdgcn_update_dpp(carry, hi, 0x138, 0xf, 0xf, false);  // wave_shr 1
  carry = __builtin_amdgcn_readlane(hi, 63);
  return GroupLane{lo, hi - lo};
}

// Workgroups are dealt to the 8 XCDs round-robin by id: workgroup bid takes item number bid / 8 of
// XCD bid % 8, each XCD a contiguous range of the items that there really are, so that the items
// on one XCD share rows and weights in that XCD's L2.  The grid holds whole rounds of 8.  -1: none.
__device__ __forceinline__ int xcd_item(int bid, int items) {
  const int x = bid & 7, i = bid >> 3, q = items >> 3, r = items & 7;
  return i < q + (x < r) ? x * q + min(x, r) + i : -1;
}

// An item of the sequence that lists, group after group, own(rows) * per items.
struct GroupItem {
  int group, row0, rows;
  int local;  // index within the group
};

// The groups as one wave sees them (every lane active): up to 64 of them are held in registers,
// more are walked again for each question.
struct Groups {
  const GroupArgs& ga;
  int M, lane, first;
  GroupLane r;
  __device__ __forceinline__ Groups(const GroupArgs& a, int M_, int lane_) : ga(a), M(M_), lane(lane_), first(0) {
    if (!ga.offsets) {
      r = GroupLane{lane ? M : 0, lane ? 0 : M};
      return;
    }
    first = clamp_offset(ga.offsets[0], M);
    int carry = first;
    r = group_lane(ga, M, 0, lane, carry);
  }
  __device__ __forceinline__ bool held() const { return ga.groups <= 64; }
  template <class F>
  __device__ __forceinline__ int total(F own) const {
    if (held()) return __builtin_amdgcn_readlane(scan_add(own(r.rows)), 63);
    int carry = first, sum = 0;
    for (int base = 0; base < ga.groups; base += 64)
      sum += __builtin_amdgcn_readlane(scan_add(own(group_lane(ga, M, base, lane, carry).rows)), 63);
    return sum;
  }
  // Item t, which is below total(own) * per.
  template <class F>
  __device__ __forceinline__ GroupItem find(F own, int per, int t) const {
    GroupLane q = r;
    int n = own(q.rows), end = scan_add(n), base = 0;
    if (!held()) {
      int carry = first, before = 0;
      for (;; base += 64) {
        q = group_lane(ga, M, base, lane, carry);
        n = own(q.rows);
        end = before + scan_add(n);
        before = __builtin_amdgcn_readlane(end, 63);
        if (before * per > t || base + 64 >= ga.groups) break;
      }
    }
    const int l = __builtin_ctzll(__ballot(end * per > t) | (1ull << 63));
    return GroupItem{base + l, __builtin_amdgcn_readlane(q.row0, l), __builtin_amdgcn_readlane(q.rows, l),
                     t - __builtin_amdgcn_readlane(end - n, l) * per};
  }
  __device__ __forceinline__ GroupLane rows_of(int g) const {
    GroupLane q = r;
    if (!held()) {
      int carry = first;
      for (int base = 0; base <= g; base += 64) q = group_lane(ga, M, base, lane, carry);
    }
    return GroupLane{__builtin_amdgcn_readlane(q.row0, g & 63), __builtin_amdgcn_readlane(q.rows, g & 63)};
  }
  // The j-th group in falling order of the power of two below its rows (up to 64 groups; more keep
  // their own order): work whose time goes with the rows is best begun with the longest.
  __device__ __forceinline__ int by_size(int j) const {
    if (!held()) return j;
    const int size = lane < ga.groups ? 32 - __clz(r.rows) : -1;
    for (int c = 32 - __clz(M); c >= 0; --c) {
      const uint64_t m = __ballot(size == c);
      const int n = __popcll(m);
      if (j < n) {
        const int rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
        return __builtin_ctzll(__ballot(size == c && rank == j) | (1ull << 63));
      }
      j -= n;
    }
    return j;  // past the last group
  }
};

// Item `bid` of the sequence with ceil(rows / bm) * per items a group, dealt out by xcd_item; group
// -1: none (the grid is sized for the worst case).
__device__ __forceinline__ GroupItem group_item(const GroupArgs& ga, int M, int bm, int per, int bid, int lane) {
  const Groups gs(ga, M, lane);
  auto own = [bm](int rows) { return (rows + bm - 1) / bm; };
  const int t = xcd_item(bid, gs.total(own) * per);
  return t < 0 ? GroupItem{-1, 0, 0, 0} : gs.find(own, per, t);
}
inline int64_t whole_rounds(int64_t items) { return (items + 7) / 8 * 8; }

// Moves the arguments of a product on to one group: its rows of A and C (and their scales), its
// B, bias and column scales; with MX its block scales.
template <int ES, int CES, bool MX = false>
__device__ __forceinline__ void enter_group(GemmParams& p, const GroupArgs& ga, int group, int row0, int rows) {
  p.A = reinterpret_cast<const uint8_t*>(p.A) + (int64_t)row0 * p.lda * ES;
  p.B = reinterpret_cast<const uint8_t*>(p.B) + (int64_t)group * ga.stride_b * ES;
  p.C = reinterpret_cast<uint8_t*>(p.C) + (int64_t)row0 * p.ldc * CES;
  p.M = rows;
  if (p.bias) p.bias += (int64_t)group * p.N;
  if (p.ra) p.ra += row0;
  if (p.rb) p.rb += (int64_t)group * p.N;
  if constexpr (MX) {
    p.sa += (int64_t)row0 * p.ldsa;
    p.sb += (int64_t)group * ga.stride_sb;
  }
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

// The bias gradient, dbias_g[n] = the sum of D's rows of group g, is the work of the first
// workgroups of the weight gradient's grid (64 columns of one group each), so that it runs beside
// the products and costs no launch.  Lane l sums 8 columns of every (threads / 8)-th row; the
// lanes of a wave meet by shuffles and the waves in LDS, in an order that depends on the group's
// size alone.  It takes 5 of the 87 us of 8 gradients of 4096 x 2048 from 4096 rows.
struct BiasGrad {
  const void* D;
  int64_t ldd;
  int N, blocks_n, blocks;  // blocks: all of them, a whole number of rounds of 8 (0: none)
  float* out;
};

}  // namespace tgemm
