// Products grouped by expert on the matrix-core tiles of mfma.hpp (gfx950 only): a workgroup finds
// its group from the offsets, moves the arguments on to it and runs one tile as any product does.
#pragma once

#include "grouped.hpp"
#include "mfma.hpp"

namespace tgemm {

// Tiles of the launchers below.
enum GroupedTile : int { GT_ANY = 0, GT_64 = 1, GT_128 = 2, GT_256 = 3, GT_64_DEEP = 4, GT_ANY_DEEP = 5 };

template <class C>
__device__ __forceinline__ void grouped_rows_tile(GemmParams& p, const GroupArgs& ga, uint8_t* smem) {
  const GroupItem it = group_item(ga, p.M, C::BM, p.tiles_n, workgroup(ga), threadIdx.x & 63);
  if (it.group < 0) return;
  enter_group<C::ES, DTypeInfo<C::CT>::bytes, C::MX>(p, ga, it.group, it.row0, it.rows);
  mfma_tile<C>(p, SkSeg{}, smem, tile_pos(it.local, (it.rows + C::BM - 1) / C::BM, p.tiles_n));
}

template <class C>
__global__ __launch_bounds__(C::NT) void grouped_rows_kernel(GemmParams p, GroupArgs ga) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS_BYTES];
  grouped_rows_tile<C>(p, ga, smem);
}
// The same with the registers of two waves a SIMD at most.
template <class C>
__global__ __launch_bounds__(C::NT, 2) void grouped_rows_two_kernel(GemmParams p, GroupArgs ga) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS_BYTES];
  grouped_rows_tile<C>(p, ga, smem);
}

// 256 x 256 tiles (F) with 128 x 128 ones (Q) where the large would waste the chip:
//  * a group's last rows, if at most 128 of them are left over, are tiles of 128 rows;
//  * of the large tiles that do not fill a whole round of the compute units, each is split into
//    four if the round gets shorter that way.
// A small tile takes about 0.4 of a large one's time (bf16, K = 2048: 22 and 54 us), which decides:
// the time of the last rounds is estimated both ways in tenths of a large tile, small ones filling
// the holes of a started round two to a hole.  Large tiles come first, so that the small ones end
// the launch.  Measured (4096 rows over 8 groups, N 4096, K 2048, bf16; 8190 over 16, N 2048, K
// 4096, fp16): 115 and 222 us with large tiles alone, 86 to 88 and 161 to 171 mixed.
__host__ __device__ __forceinline__ int large_rows(int rows) { return (int)(((int64_t)rows + 127) >> 8); }
__host__ __device__ __forceinline__ int small_rows(int rows) { return (rows & 255) && (rows & 255) <= 128 ? 1 : 0; }
// How many of nl large tiles to split, beside ns small ones.
__host__ __device__ __forceinline__ int tiles_to_split(int nl, int ns, int cus) {
  const int rounds = nl / cus, rest = nl - rounds * cus;
  const int over = ns - (rest ? 2 * (cus - rest) : 0);
  const int whole = 10 * (rounds + (rest > 0)) + 4 * (((over > 0 ? over : 0) + cus - 1) / cus);
  const int apart = 10 * rounds + 4 * (int)((ns + 4 * (int64_t)rest + cus - 1) / cus);
  return apart < whole ? rest : 0;
}

// `workers`: the workgroups (a whole number of rounds of 8) that share out the small tiles.  A
// workgroup without work still has to wait for its LDS, so the grid holds no more of them than the
// worst case of the large tiles asks for.
template <class F, class Q>
__global__ __launch_bounds__(512) void grouped_rows_mixed_kernel(const GemmParams p0, GroupArgs ga, int cus, int workers) {
  static_assert(F::NT == 512 && Q::NT == 512 && F::BM == 256 && Q::BM == 128, "two tiles of one workgroup size");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[F::LDS_BYTES > Q::LDS_BYTES ? F::LDS_BYTES : Q::LDS_BYTES];
  const Groups gs(ga, p0.M, threadIdx.x & 63);
  const int tn = (int)(((int64_t)p0.N + 255) >> 8), tn_small = (int)(((int64_t)p0.N + 127) >> 7);
  const int nl = gs.total(large_rows) * tn, ns = gs.total(small_rows) * tn_small;
  const int split = __builtin_amdgcn_readfirstlane(tiles_to_split(nl, ns, cus)), kept = nl - split;
  const int first_small = (kept + 7) & ~7, bid = workgroup(ga);
  if (bid < first_small) {
    const int t = xcd_item(bid, kept);
    if (t < 0) return;
    const GroupItem it = gs.find(large_rows, tn, t);
    GemmParams p = p0;
    enter_group<F::ES, DTypeInfo<F::CT>::bytes, F::MX>(p, ga, it.group, it.row0, it.rows);
    mfma_tile<F>(p, SkSeg{}, smem, tile_pos(it.local, large_rows(it.rows), tn));
    return;
  }
  if (bid - first_small >= workers) return;
  const int pieces = 4 * split + ns;
  for (int base = 0; base < pieces; base += workers) {
    const int i = xcd_item(bid - first_small, min(workers, pieces - base));
    if (i < 0) return;
    const int t = base + i;
    GroupItem it;
    TilePos at;
    if (t < 4 * split) {
      it = gs.find(large_rows, tn, kept + (t >> 2));
      at = tile_pos(it.local, large_rows(it.rows), tn);
      at = TilePos{2 * at.tm + (t & 1), 2 * at.tn + ((t >> 1) & 1)};
    } else {
      it = gs.find(small_rows, tn_small, t - 4 * split);
      at = TilePos{2 * large_rows(it.rows), it.local};
    }
    if (128 * at.tm >= it.rows || 128 * at.tn >= p0.N) continue;  // a quarter past the edge
    if (base) __syncthreads();  // the last tile's output staging has been read
    GemmParams p = p0;
    enter_group<Q::ES, DTypeInfo<Q::CT>::bytes, Q::MX>(p, ga, it.group, it.row0, it.rows);
    mfma_tile<Q>(p, SkSeg{}, smem, at);
  }
}

template <int DT, int NT>
__device__ __forceinline__ void bias_tile(const BiasGrad& b, const GroupArgs& ga, int M, int bid) {
  constexpr int NW = NT / 64;
  __shared__ float part[NW][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = bid / b.blocks_n;
  if (g >= ga.groups) return;
  const int n0 = bid % b.blocks_n * 64, n = n0 + 8 * (lane & 7);
  const GroupLane r = Groups(ga, M, lane).rows_of(g);
  float s[8] = {};
  const uint16_t* const D = reinterpret_cast<const uint16_t*>(b.D) + (int64_t)r.row0 * b.ldd;
  auto add = [&](u32x4 v) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = (v[e >> 1] >> (16 * (e & 1))) & 0xffffu;
      s[e] += DT == BF16 ? bf16_bits_to_float(h) : f16_bits_to_float(h);
    }
  };
  if (n + 8 <= b.N) {
    constexpr int STEP = NT / 8;
    int i = tid >> 3;
    for (; i + 3 * STEP < r.rows; i += 4 * STEP) {  // four loads in flight
      u32x4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) __builtin_memcpy(&v[u], D + (int64_t)(i + u * STEP) * b.ldd + n, 16);
#pragma unroll
      for (int u = 0; u < 4; ++u) add(v[u]);
    }
    for (; i < r.rows; i += STEP) {
      u32x4 v;
      __builtin_memcpy(&v, D + (int64_t)i * b.ldd + n, 16);
      add(v);
    }
  } else if (n < b.N) {
    for (int i = tid >> 3; i < r.rows; i += NT / 8)
      add(load_partial<2>(reinterpret_cast<const uint8_t*>(D + (int64_t)i * b.ldd + n), b.N - n));
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int d = 8; d < 64; d <<= 1) s[e] += __shfl_xor(s[e], d);
  if (lane < 8)
#pragma unroll
    for (int e = 0; e < 8; ++e) part[wave][8 * lane + e] = s[e];
  __syncthreads();
  if (tid < 64 && n0 + tid < b.N) {
    float t = part[0][tid];
#pragma unroll
    for (int w = 1; w < NW; ++w) t += part[w][tid];
    b.out[(int64_t)g * b.N + n0 + tid] = t;
  }
}

// The weight gradient: p.M x p.N is the gradient as stored, p.A and p.B the rows it is the product
// of, p.K all rows.  xcd: the tiles of each group are dealt out to the XCDs in contiguous ranges
// (a group's rows decide its tiles' time, so whole groups are never given to one XCD); otherwise,
// with too few tiles in a group for that, tile after tile.  Groups with the most rows come first
// (8 groups of 4096 x 2048 bf16 from 4096 uneven rows: 90 us in their own order, 84 so).
// What bounds it with few rows to a group is the writing of the gradient, which the products do not
// hide: those 8 groups take 30 us with no rows at all and 0.1 us more for each row of a group (53 us
// for 512, 1.3 PFLOP/s).  16 groups of 4096 x 2048 from 16383 rows in fp32: 315 to 326 us, 0.5 GB
// written.  With beta C is read as the sums are laid out, 16 bytes of each of 32 rows an instruction,
// and nothing hides it: these two take 132 and 418 us.
template <class C>
__global__ __launch_bounds__(C::NT) void grouped_wgrad_kernel(GemmParams p, GroupArgs ga, BiasGrad b, int xcd) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS_BYTES];
  int bid = workgroup(ga);
  if (bid < b.blocks) {
    bias_tile<C::DT, C::NT>(b, ga, p.K, bid);
    return;
  }
  bid -= b.blocks;
  const int tiles = p.tiles_m * p.tiles_n;
  int g, local;
  if (xcd) {
    const int per = (tiles + 7) >> 3;
    g = (bid >> 3) / per;
    local = (bid & 7) * per + (bid >> 3) % per;
  } else {
    g = bid / tiles;
    local = bid % tiles;
  }
  if (g >= ga.groups || local >= tiles) return;
  // in scalar registers, as the tile's addresses have to be
  local = __builtin_amdgcn_readfirstlane(local);
  const Groups gs(ga, p.K, threadIdx.x & 63);
  g = __builtin_amdgcn_readfirstlane(gs.by_size(__builtin_amdgcn_readfirstlane(g)));
  const GroupLane r = gs.rows_of(g);
  enter_group_wgrad<C::ES, DTypeInfo<C::CT>::bytes>(p, ga, g, r.row0, r.rows);
  mfma_tile<C>(p, SkSeg{}, smem, tile_pos(local, p.tiles_m, p.tiles_n));
}

template <class C, bool TWO = false>
hipError_t launch_rows_cfg(GemmParams p, GroupArgs ga, hipStream_t s) {
  p.tiles_n = (p.N + C::BN - 1) / C::BN;
  const int64_t grid = whole_rounds(max_row_tiles(p.M, ga.groups, C::BM) * p.tiles_n);
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  if (!C::UNAL) {  // the last K tile's fix-ups, as for a single product
    constexpr int CE = 16 / C::ES;
    if (p.K % C::BKE) p.epi |= FIX_A;
    if (C::B_MN ? p.N % CE : p.K % C::BKE) p.epi |= FIX_B;
  }
  return launch_in_slices(grid, C::NT, [&](int64_t first, unsigned n) {
    ga.first = (int)first;
    if constexpr (TWO) hipLaunchKernelGGL((grouped_rows_two_kernel<C>), dim3(n), dim3(C::NT), 0, s, p, ga);
    else hipLaunchKernelGGL((grouped_rows_kernel<C>), dim3(n), dim3(C::NT), 0, s, p, ga);
  });
}

template <class F, class Q>
hipError_t launch_mixed_cfg(GemmParams p, GroupArgs ga, int cus, hipStream_t s) {
  const int64_t tn = ((int64_t)p.N + 255) / 256, tn_small = ((int64_t)p.N + 127) / 128;
  int64_t large, small = cus;
  if (ga.offsets) {
    const int64_t live = ga.groups < p.M ? ga.groups : p.M;
    large = (p.M + 127 * live) / 256 * tn;
  } else {  // one group: exactly
    const int64_t nl = large_rows(p.M) * tn, ns = small_rows(p.M) * tn_small;
    const int split = tiles_to_split((int)nl, (int)ns, cus);
    large = nl - split;
    small = 4 * (int64_t)split + ns;
  }
  if (small > cus) small = cus;
  const int64_t workers = whole_rounds(small), grid = whole_rounds(large) + workers;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  constexpr int CE = 16 / F::ES;
  static_assert(F::BKE == Q::BKE, "one K tile");
  if (p.K % F::BKE) p.epi |= FIX_A;
  if (F::B_MN ? p.N % CE : p.K % F::BKE) p.epi |= FIX_B;
  return launch_in_slices(grid, 512, [&](int64_t first, unsigned n) {
    ga.first = (int)first;
    hipLaunchKernelGGL((grouped_rows_mixed_kernel<F, Q>), dim3(n), dim3(512), 0, s, p, ga, cus, (int)workers);
  });
}

template <class C>
hipError_t launch_wgrad_cfg(GemmParams p, GroupArgs ga, BiasGrad b, hipStream_t s) {
  p.tiles_m = (p.M + C::BM - 1) / C::BM;
  p.tiles_n = (p.N + C::BN - 1) / C::BN;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  const int xcd = tiles % 8 == 0 || tiles >= 64;
  b.blocks_n = (b.N + 63) / 64;
  const int64_t blocks = b.out ? whole_rounds((int64_t)b.blocks_n * ga.groups) : 0;
  const int64_t grid = blocks + (xcd ? whole_rounds(tiles) : tiles) * ga.groups;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  b.blocks = (int)blocks;
  if (!C::UNAL) {
    constexpr int CE = 16 / C::ES;
    if (p.M % CE) p.epi |= FIX_A;
    if (p.N % CE) p.epi |= FIX_B;
  }
  return launch_in_slices(grid, C::NT, [&](int64_t first, unsigned n) {
    ga.first = (int)first;
    hipLaunchKernelGGL((grouped_wgrad_kernel<C>), dim3(n), dim3(C::NT), 0, s, p, ga, b, xcd);
  });
}

// MfmaCfg of a tile (B_MN / A_MN: stored contiguous along N / M).
//  * any alignment: each K tile waits for its loads and its LDS stores in turn; deep, four groups
//    of waves split K, for when a compute unit has one tile at most (37 x 4104 x 4112 in 8 bits 37
//    against 78 us, but 4096^3 226 against 147);
//  * 64 x 64: two groups split K; deep, four stages each (one workgroup a compute unit) instead
//    of two (two workgroups), for when there is no second tile to run beside the first: 1584 rows
//    over 2 groups, N 80, K 5832, bf16, 31 against 40 us, but 545 tiles 39 against 33;
//  * 128 x 128: four stages, eight waves: at K = 2048 (bf16) a tile takes 22 us, against 26 with K
//    split between two groups of four waves with two stages each.
template <int DT, int CT, bool A_MN, bool B_MN, int TILE> struct GroupedCfg;
template <int DT, int CT, bool A_MN, bool B_MN> struct GroupedCfg<DT, CT, A_MN, B_MN, GT_ANY> {
  using T = MfmaCfg<DT, 64, 2, 2, A_MN, B_MN, 2, DT, false, 0, 1, 0, 1, CT, true, true>;
};
template <int DT, int CT, bool A_MN, bool B_MN> struct GroupedCfg<DT, CT, A_MN, B_MN, GT_ANY_DEEP> {
  using T = MfmaCfg<DT, 64, 2, 2, A_MN, B_MN, 2, DT, false, 0, 4, 0, 1, CT, true, true>;
};
template <int DT, int CT, bool A_MN, bool B_MN> struct GroupedCfg<DT, CT, A_MN, B_MN, GT_64> {
  using T = MfmaCfg<DT, 64, 2, 2, A_MN, B_MN, 2, DT, false, 0, 2, 0, 1, CT, true>;
};
template <int DT, int CT, bool A_MN, bool B_MN> struct GroupedCfg<DT, CT, A_MN, B_MN, GT_64_DEEP> {
  using T = MfmaCfg<DT, 64, 2, 2, A_MN, B_MN, 4, DT, false, 0, 2, 0, 1, CT, true>;
};
template <int DT, int CT, bool A_MN, bool B_MN> struct GroupedCfg<DT, CT, A_MN, B_MN, GT_128> {
  using T = MfmaCfg<DT, 128, 2, 4, A_MN, B_MN, 4, DT, false, 0, 1, 0, 1, CT, true>;
};
template <int DT, int CT, bool A_MN, bool B_MN> struct GroupedCfg<DT, CT, A_MN, B_MN, GT_256> {
  using T = MfmaCfg<DT, 256, 2, 4, A_MN, B_MN, 2, DT, false, 0, 1, 0, 1, CT, true>;
};

template <int DT, int CT, bool B_MN>
hipError_t launch_mixed_type(const GemmParams& p, const GroupArgs& ga, int cus, hipStream_t s) {
  return launch_mixed_cfg<typename GroupedCfg<DT, CT, false, B_MN, GT_256>::T,
                          typename GroupedCfg<DT, CT, false, B_MN, GT_128>::T>(p, ga, cus, s);
}

template <int DT, int CT, bool B_MN>
hipError_t launch_rows_layout(const GemmParams& p, const GroupArgs& ga, int tile, int cus, hipStream_t s) {
  switch (tile) {
    case GT_ANY: return launch_rows_cfg<typename GroupedCfg<DT, CT, false, B_MN, GT_ANY>::T>(p, ga, s);
    case GT_ANY_DEEP: return launch_rows_cfg<typename GroupedCfg<DT, CT, false, B_MN, GT_ANY_DEEP>::T>(p, ga, s);
    case GT_64: return launch_rows_cfg<typename GroupedCfg<DT, CT, false, B_MN, GT_64>::T>(p, ga, s);
    case GT_64_DEEP: return launch_rows_cfg<typename GroupedCfg<DT, CT, false, B_MN, GT_64_DEEP>::T>(p, ga, s);
    case GT_128: return launch_rows_cfg<typename GroupedCfg<DT, CT, false, B_MN, GT_128>::T>(p, ga, s);
    case GT_256: return launch_mixed_type<DT, CT, B_MN>(p, ga, cus, s);
    default: return hipErrorInvalidValue;
  }
}

template <int DT, int CT>
hipError_t launch_rows_type(const GemmParams& p, const GroupArgs& ga, bool b_mn, int tile, int cus, hipStream_t s) {
  return b_mn ? launch_rows_layout<DT, CT, true>(p, ga, tile, cus, s) : launch_rows_layout<DT, CT, false>(p, ga, tile, cus, s);
}

// The same tiles in MXFP4 (both operands packed along K; K, lda and ldb in bytes; K is not split).  Their
// block scales are staged beside the data for two K tiles at a time.
//  * 64 x 64: at the rate of the memory with few rows to a group (64 rows over 32 groups of 2048 x 2048 14 us,
//    71 MB; streamed 18); deep, three stages instead of two, for few tiles of a long K (16 x 28672 x 8192 31
//    us against 35, but 384 x 4096 x 4096 13.7 against 13.1);
//  * 128 x 128: four waves and two stages, so that two workgroups share a compute unit and one's products
//    hide the other's copies and output (4096 rows over 32 groups of 2048 x 2048 24 us; eight waves with
//    three stages, as the mixed kernel has to have them, 30).
template <int CT, int TILE> struct GroupedMxCfg;
template <int CT> struct GroupedMxCfg<CT, GT_64> {
  using T = MfmaCfg<E2M1, 64, 2, 2, false, false, 2, E2M1, true, 0, 1, 0, 1, CT, true>;
};
template <int CT> struct GroupedMxCfg<CT, GT_64_DEEP> {
  using T = MfmaCfg<E2M1, 64, 2, 2, false, false, 3, E2M1, true, 0, 1, 0, 1, CT, true>;
};
template <int CT> struct GroupedMxCfg<CT, GT_128> {
  using T = MfmaCfg<E2M1, 128, 2, 2, false, false, 2, E2M1, true, 0, 1, 0, 1, CT, true>;
};
template <int CT> struct GroupedMxCfg<CT, GT_256> {
  using T = MfmaCfg<E2M1, 256, 2, 4, false, false, 2, E2M1, true, 0, 1, 0, 1, CT, true>;
  using Small = MfmaCfg<E2M1, 128, 2, 4, false, false, 3, E2M1, true, 0, 1, 0, 1, CT, true>;
};

template <int CT>
hipError_t launch_mx_type(const GemmParams& p, const GroupArgs& ga, int tile, int cus, hipStream_t s) {
  using Large = GroupedMxCfg<CT, GT_256>;
  switch (tile) {
    case GT_64: return launch_rows_cfg<typename GroupedMxCfg<CT, GT_64>::T>(p, ga, s);
    case GT_64_DEEP: return launch_rows_cfg<typename GroupedMxCfg<CT, GT_64_DEEP>::T>(p, ga, s);
    case GT_128: return launch_rows_cfg<typename GroupedMxCfg<CT, GT_128>::T, true>(p, ga, s);
    case GT_256: return launch_mixed_cfg<typename Large::T, typename Large::Small>(p, ga, cus, s);
    default: return hipErrorInvalidValue;
  }
}

template <int DT, int CT>
hipError_t launch_wgrad_type(const GemmParams& p, const GroupArgs& ga, const BiasGrad& b, int tile, hipStream_t s) {
  switch (tile) {
    case GT_ANY: return launch_wgrad_cfg<typename GroupedCfg<DT, CT, true, true, GT_ANY>::T>(p, ga, b, s);
    case GT_ANY_DEEP: return launch_wgrad_cfg<typename GroupedCfg<DT, CT, true, true, GT_ANY_DEEP>::T>(p, ga, b, s);
    case GT_64_DEEP: return launch_wgrad_cfg<typename GroupedCfg<DT, CT, true, true, GT_64_DEEP>::T>(p, ga, b, s);
    case GT_64: return launch_wgrad_cfg<typename GroupedCfg<DT, CT, true, true, GT_64>::T>(p, ga, b, s);
    case GT_128: return launch_wgrad_cfg<typename GroupedCfg<DT, CT, true, true, GT_128>::T>(p, ga, b, s);
    case GT_256: return launch_wgrad_cfg<typename GroupedCfg<DT, CT, true, true, GT_256>::T>(p, ga, b, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tgemm
