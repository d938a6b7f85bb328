// Products grouped by expert on the matrix-core tiles of mfma.hpp (gfx950 only): a workgroup finds
// its group from the offsets, moves the arguments on to it and runs one tile as any product does.
#pragma once

#include "grouped.hpp"
#include "mfma.hpp"

namespace tgemm {

// Tiles of the launchers below.
enum GroupedTile : int { GT_ANY = 0, GT_64 = 1, GT_128 = 2, GT_256x128 = 3, GT_256 = 4 };

template <class C>
__global__ __launch_bounds__(C::NT) void grouped_rows_kernel(GemmParams p, GroupArgs ga) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS_BYTES];
  const GroupItem it = group_item(ga, p.M, C::BM, p.tiles_n, (int)blockIdx.x, threadIdx.x & 63);
  if (it.group < 0) return;
  enter_group<C::ES, DTypeInfo<C::CT>::bytes>(p, ga, it.group, it.row0, it.rows);
  mfma_tile<C>(p, SkSeg{}, smem, tile_pos(it.local, (it.rows + C::BM - 1) / C::BM, p.tiles_n));
}

// 256 x 256 tiles (F) with 128 x 128 ones (Q) where the large would waste the chip:
//  * a group's last rows, if at most 128 of them are left over, are tiles of 128 rows;
//  * of the large tiles that do not fill a whole round of the compute units, each is split into
//    four if the round gets shorter that way.  A split tile costs about 0.3 of a large one (its K
//    loop is shared by two groups of waves), which decides: the time of the last rounds is
//    estimated both ways in tenths of a large tile, small ones filling the holes of a started
//    round three to a hole.
// Large tiles come first, so that the small ones end the launch.
template <class F, class Q>
__global__ __launch_bounds__(512) void grouped_rows_mixed_kernel(GemmParams p, GroupArgs ga, int cus) {
  static_assert(F::NT == 512 && Q::NT == 512 && F::BM == 256 && Q::BM == 128, "two tiles of one workgroup size");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[F::LDS_BYTES > Q::LDS_BYTES ? F::LDS_BYTES : Q::LDS_BYTES];
  const Groups gs(ga, p.M, threadIdx.x & 63);
  auto large = [](int rows) { return (int)(((int64_t)rows + 127) >> 8); };
  auto small = [](int rows) { return (rows & 255) && (rows & 255) <= 128 ? 1 : 0; };
  const int tn = (p.N + 255) >> 8, tn_small = (p.N + 127) >> 7;
  const int nl = gs.total(large) * tn, ns = gs.total(small) * tn_small;
  const int rounds = nl / cus, rest = nl - rounds * cus;
  const int whole = 10 * (rounds + (rest > 0)) + 3 * ((max(0, ns - (rest ? 3 * (cus - rest) : 0)) + cus - 1) / cus);
  const int apart = 10 * rounds + 3 * ((ns + 4 * rest + cus - 1) / cus);
  const int split = __builtin_amdgcn_readfirstlane(apart < whole ? rest : 0), kept = nl - split;
  int bid = (int)blockIdx.x;
  const int first_small = (kept + 7) & ~7;
  if (bid < first_small) {
    const int t = xcd_item(bid, kept);
    if (t < 0) return;
    const GroupItem it = gs.find(large, tn, t);
    enter_group<F::ES, DTypeInfo<F::CT>::bytes>(p, ga, it.group, it.row0, it.rows);
    mfma_tile<F>(p, SkSeg{}, smem, tile_pos(it.local, large(it.rows), tn));
    return;
  }
  const int t = xcd_item(bid - first_small, 4 * split + ns);
  if (t < 0) return;
  GroupItem it;
  TilePos at;
  if (t < 4 * split) {
    it = gs.find(large, tn, kept + (t >> 2));
    at = tile_pos(it.local, large(it.rows), tn);
    at = TilePos{2 * at.tm + (t & 1), 2 * at.tn + ((t >> 1) & 1)};
    if (128 * at.tm >= it.rows || 128 * at.tn >= p.N) return;
  } else {
    it = gs.find(small, tn_small, t - 4 * split);
    at = TilePos{2 * large(it.rows), it.local};
  }
  enter_group<Q::ES, DTypeInfo<Q::CT>::bytes>(p, ga, it.group, it.row0, it.rows);
  mfma_tile<Q>(p, SkSeg{}, smem, at);
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
// with too few tiles in a group for that, tile after tile.
template <class C>
__global__ __launch_bounds__(C::NT) void grouped_wgrad_kernel(GemmParams p, GroupArgs ga, BiasGrad b, int xcd) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS_BYTES];
  int bid = (int)blockIdx.x;
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

template <class C>
hipError_t launch_rows_cfg(GemmParams p, const GroupArgs& ga, hipStream_t s) {
  p.tiles_n = (p.N + C::BN - 1) / C::BN;
  const int64_t grid = whole_rounds(max_row_tiles(p.M, ga.groups, C::BM) * p.tiles_n);
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  if (!C::UNAL) {  // the last K tile's fix-ups, as for a single product
    constexpr int CE = 16 / C::ES;
    if (p.K % C::BKE) p.epi |= FIX_A;
    if (C::B_MN ? p.N % CE : p.K % C::BKE) p.epi |= FIX_B;
  }
  hipLaunchKernelGGL((grouped_rows_kernel<C>), dim3((unsigned)grid), dim3(C::NT), 0, s, p, ga);
  return hipGetLastError();
}

template <class F, class Q>
hipError_t launch_mixed_cfg(GemmParams p, const GroupArgs& ga, int cus, hipStream_t s) {
  const int64_t rows = max_row_tiles(p.M, ga.groups, 256), live = ga.groups < p.M ? ga.groups : p.M;
  const int64_t grid = whole_rounds(rows * ((p.N + 255) / 256)) +
                       whole_rounds(4 * (int64_t)cus + live * ((p.N + 127) / 128));
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  constexpr int CE = 16 / F::ES;
  static_assert(F::BKE == Q::BKE, "one K tile");
  if (p.K % F::BKE) p.epi |= FIX_A;
  if (F::B_MN ? p.N % CE : p.K % F::BKE) p.epi |= FIX_B;
  hipLaunchKernelGGL((grouped_rows_mixed_kernel<F, Q>), dim3((unsigned)grid), dim3(512), 0, s, p, ga, cus);
  return hipGetLastError();
}

template <class C>
hipError_t launch_wgrad_cfg(GemmParams p, const GroupArgs& ga, BiasGrad b, hipStream_t s) {
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
  if (grid > 0) hipLaunchKernelGGL((grouped_wgrad_kernel<C>), dim3((unsigned)grid), dim3(C::NT), 0, s, p, ga, b, xcd);
  return hipGetLastError();
}

// MfmaCfg of a tile: B_MN / A_MN: stored contiguous along N / M.
template <int DT, int CT, bool A_MN, bool B_MN, int TILE>
struct GroupedCfg {
  using T = typename std::conditional<
      TILE == GT_ANY, MfmaCfg<DT, 64, 2, 2, A_MN, B_MN, 2, DT, false, 0, 1, 0, 1, CT, true, true>,
      typename std::conditional<
          TILE == GT_64, MfmaCfg<DT, 64, 2, 2, A_MN, B_MN, 2, DT, false, 0, 2, 0, 1, CT, true>,
          typename std::conditional<
              TILE == GT_128, MfmaCfg<DT, 128, 2, 2, A_MN, B_MN, 2, DT, false, 0, 2, 0, 1, CT, true>,
              typename std::conditional<
                  TILE == GT_256x128, MfmaCfg<DT, 256, 4, 2, A_MN, B_MN, 2, DT, false, 0, 1, 128, 1, CT, true>,
                  MfmaCfg<DT, 256, 2, 4, A_MN, B_MN, 2, DT, false, 0, 1, 0, 1, CT, true>>::type>::type>::type>::type;
};

template <int DT, int CT, bool B_MN>
hipError_t launch_mixed_type(const GemmParams& p, const GroupArgs& ga, int cus, hipStream_t s) {
  return launch_mixed_cfg<typename GroupedCfg<DT, CT, false, B_MN, GT_256>::T,
                          typename GroupedCfg<DT, CT, false, B_MN, GT_128>::T>(p, ga, cus, s);
}

template <int DT, int CT>
hipError_t launch_rows_type(const GemmParams& p, const GroupArgs& ga, bool b_mn, int tile, int cus, hipStream_t s) {
  switch (tile * 2 + b_mn) {
    case GT_ANY * 2: return launch_rows_cfg<typename GroupedCfg<DT, CT, false, false, GT_ANY>::T>(p, ga, s);
    case GT_ANY * 2 + 1: return launch_rows_cfg<typename GroupedCfg<DT, CT, false, true, GT_ANY>::T>(p, ga, s);
    case GT_64 * 2: return launch_rows_cfg<typename GroupedCfg<DT, CT, false, false, GT_64>::T>(p, ga, s);
    case GT_64 * 2 + 1: return launch_rows_cfg<typename GroupedCfg<DT, CT, false, true, GT_64>::T>(p, ga, s);
    case GT_128 * 2: return launch_rows_cfg<typename GroupedCfg<DT, CT, false, false, GT_128>::T>(p, ga, s);
    case GT_128 * 2 + 1: return launch_rows_cfg<typename GroupedCfg<DT, CT, false, true, GT_128>::T>(p, ga, s);
    case GT_256x128 * 2: return launch_rows_cfg<typename GroupedCfg<DT, CT, false, false, GT_256x128>::T>(p, ga, s);
    case GT_256x128 * 2 + 1: return launch_rows_cfg<typename GroupedCfg<DT, CT, false, true, GT_256x128>::T>(p, ga, s);
    case GT_256 * 2: return launch_mixed_type<DT, CT, false>(p, ga, cus, s);
    case GT_256 * 2 + 1: return launch_mixed_type<DT, CT, true>(p, ga, cus, s);
    default: return hipErrorInvalidValue;
  }
}

template <int DT, int CT>
hipError_t launch_wgrad_type(const GemmParams& p, const GroupArgs& ga, const BiasGrad& b, int tile, hipStream_t s) {
  switch (tile) {
    case GT_ANY: return launch_wgrad_cfg<typename GroupedCfg<DT, CT, true, true, GT_ANY>::T>(p, ga, b, s);
    case GT_64: return launch_wgrad_cfg<typename GroupedCfg<DT, CT, true, true, GT_64>::T>(p, ga, b, s);
    case GT_128: return launch_wgrad_cfg<typename GroupedCfg<DT, CT, true, true, GT_128>::T>(p, ga, b, s);
    case GT_256x128: return launch_wgrad_cfg<typename GroupedCfg<DT, CT, true, true, GT_256x128>::T>(p, ga, b, s);
    case GT_256: return launch_wgrad_cfg<typename GroupedCfg<DT, CT, true, true, GT_256>::T>(p, ga, b, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tgemm
