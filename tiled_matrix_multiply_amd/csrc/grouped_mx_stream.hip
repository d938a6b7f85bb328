// Products by expert in MXFP4 for few rows per group (decoding), where the weights are read once and
// nothing else matters; and for any alignment (gfx950 only).
//
// As the streaming kernel of the wider types: a workgroup owns 16 NF columns of one group and up to 16 MF
// of its rows, its four waves share out K and meet in LDS at the end, in wave order, and weights and rows
// go straight from global memory into the registers of scaled 16 x 16 x 128 matrix instructions.  Lane l
// of a fragment holds row (column) l % 16 and the 32 elements k = 32 (l / 16) .. + 31 of a step of 128, 16
// bytes, with the one scale that belongs to them.  A unit is U steps; its 4 U scale bytes of a row come
// in one load, the same for the four lanes of the row, and each lane moves its own byte of a step down.
//
// Up to 8 rows the weights' bytes bound it (1 x 28672 x 8192 24.8 us, 5.0 TB/s; 32 rows over 64 groups of 1024 x
// 2048 9.2, 28 MB), with more the caches' rate: every tile reads its rows and columns again (48 x 4096 x 8192, 256
// tiles of 32 x 32, 12.2 us, 67 MB).
#include <type_traits>

#include "grouped.hpp"

namespace tgemm {

namespace {

typedef float x_f32x4 __attribute__((ext_vector_type(4)));
typedef int x_i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t x_u32x4 __attribute__((ext_vector_type(4)));

constexpr int NW = 4;  // waves of a workgroup

__device__ __forceinline__ x_f32x4 mma_mx(x_u32x4 x, x_u32x4 y, x_f32x4 c, int sx, int sy) {
  const x_i32x8 a = x_i32x8{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
  const x_i32x8 b = x_i32x8{(int)y[0], (int)y[1], (int)y[2], (int)y[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, 0, sx, 0, sy);
}

// K and the leading dimensions of A and B are in bytes (two elements each).
template <int NF, int MF, int U>
__global__ __launch_bounds__(64 * NW) void mx_stream_kernel(GemmParams p, GroupArgs ga, int c_type) {
  constexpr int BM = 16 * MF, BN = 16 * NF;
  __shared__ x_f32x4 part[NW][NF * MF][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const GroupItem it = group_item(ga, p.M, BM, p.tiles_n, workgroup(ga), lane);
  if (it.group < 0) return;
  if (c_type == F32) enter_group<1, 4, true>(p, ga, it.group, it.row0, it.rows);
  else enter_group<1, 2, true>(p, ga, it.group, it.row0, it.rows);
  // the row tiles of a block of columns are neighbours: they share its weights in the L2
  const int tiles_m = (p.M + BM - 1) / BM;
  const int m0 = it.local % tiles_m * BM, n0 = it.local / tiles_m * BN;
  const int q = lane >> 4, l16 = lane & 15;

  // Lane offsets (32 bits: the host keeps a row under 2^23 bytes) from a uniform base; rows and columns
  // past the edge repeat the last ones and are not stored.
  const uint8_t* const Ab = reinterpret_cast<const uint8_t*>(p.A) + (int64_t)m0 * p.lda;
  const uint8_t* const Bb = reinterpret_cast<const uint8_t*>(p.B) + (int64_t)n0 * p.ldb;
  const uint8_t* const Sa = p.sa + (int64_t)m0 * p.ldsa;
  const uint8_t* const Sb = p.sb + (int64_t)n0 * p.ldsb;
  uint32_t oa[MF], ob[NF], osa[MF], osb[NF];
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const uint32_t r = (uint32_t)min(16 * f + l16, p.M - 1 - m0);
    oa[f] = r * (uint32_t)p.lda + 16 * q;
    osa[f] = r * (uint32_t)p.ldsa;
  }
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const uint32_t r = (uint32_t)min(16 * f + l16, p.N - 1 - n0);
    ob[f] = r * (uint32_t)p.ldb + 16 * q;
    osb[f] = r * (uint32_t)p.ldsb;
  }

  // What the thread finishes at the end: items of four columns, and their bias, which would otherwise come in
  // after the sums, with nothing left to hide its way from memory.
  constexpr int ITEMS = NF * MF * 64, MINE = (ITEMS + 64 * NW - 1) / (64 * NW);
  auto item = [&](int i, int& m, int& n) {
    m = m0 + 16 * ((i >> 6) % MF) + (i & 15);
    n = n0 + 16 * ((i >> 6) / MF) + 4 * ((i & 63) >> 4);
    return (ITEMS % (64 * NW) == 0 || i < ITEMS) && m < p.M && n < p.N;
  };
  float bj[MINE][4];
#pragma unroll
  for (int t = 0; t < MINE; ++t) {
    int m, n;
    const bool live = (p.epi & EPI_BIAS) && item(threadIdx.x + 64 * NW * t, m, n);
#pragma unroll
    for (int e = 0; e < 4; ++e) bj[t][e] = live ? p.bias[min(n + e, p.N - 1)] : 0.0f;  // past the edge the last once more
  }

  struct Unit {
    x_u32x4 b[NF][U], a[MF][U];
    uint32_t sb[NF][U], sa[MF][U];
  };
  auto load = [&](int u, Unit& t) {
    const int64_t k = (int64_t)u * (64 * U);
    const uint8_t *as = Ab + k, *bs = Bb + k, *sas = Sa + (int64_t)u * (4 * U), *sbs = Sb + (int64_t)u * (4 * U);
#pragma unroll
    for (int f = 0; f < NF; ++f) {
#pragma unroll
      for (int s = 0; s < U; ++s) __builtin_memcpy(&t.b[f][s], bs + ob[f] + 64 * s, 16);
      __builtin_memcpy(t.sb[f], sbs + osb[f], 4 * U);
    }
#pragma unroll
    for (int f = 0; f < MF; ++f) {
#pragma unroll
      for (int s = 0; s < U; ++s) __builtin_memcpy(&t.a[f][s], as + oa[f] + 64 * s, 16);
      __builtin_memcpy(t.sa[f], sas + osa[f], 4 * U);
    }
  };
  x_f32x4 acc[NF][MF];
#pragma unroll
  for (int j = 0; j < NF; ++j)
#pragma unroll
    for (int f = 0; f < MF; ++f) acc[j][f] = x_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto mul = [&](const Unit& t) {
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int f = 0; f < MF; ++f)
          acc[j][f] = mma_mx(t.b[j][s], t.a[f][s], acc[j][f], (int)(t.sb[j][s] >> (8 * q)), (int)(t.sa[f][s] >> (8 * q)));
  };
  // One step of 128 elements that may end early: a lane's 32 elements are there or not (K is a whole
  // number of blocks); what is not there is 0 with scale 2^0.
  auto rest_step = [&](int s) {
    const bool there = (int64_t)s * 64 + 16 * q < p.K;
    x_u32x4 a[MF], b[NF];
    int sa[MF], sb[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      b[f] = x_u32x4{0u, 0u, 0u, 0u};
      sb[f] = 127;
      if (there) {
        __builtin_memcpy(&b[f], Bb + (int64_t)s * 64 + ob[f], 16);
        sb[f] = Sb[(int64_t)s * 4 + q + osb[f]];
      }
    }
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      a[f] = x_u32x4{0u, 0u, 0u, 0u};
      sa[f] = 127;
      if (there) {
        __builtin_memcpy(&a[f], Ab + (int64_t)s * 64 + oa[f], 16);
        sa[f] = Sa[(int64_t)s * 4 + q + osa[f]];
      }
    }
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int f = 0; f < MF; ++f) acc[j][f] = mma_mx(b[j], a[f], acc[j][f], sb[j], sa[f]);
  };

  // Whole units over the waves in turn; the steps after the last whole unit go to one wave each, before its
  // units.  A wave has one unit in flight at a time: a second one ahead would cost it the registers of two
  // more waves beside it, which hide as much (with one unit ahead, 32 rows over 64 groups of 1024 x 2048 10.2 us
  // against 8.2, 256 over 32 of 2048 x 2048 21.3 against 16.2, 1 x 16384 x 16384 37.5 against 31.5, 16 x 28672 x 8192
  // 35.7 against 37.2).
  const int steps = (int)(((int64_t)p.K + 63) / 64), units = p.K / (64 * U), first = units * U;
  for (int s = first + wave; s < steps; s += NW) rest_step(s);
  for (int b = wave; b < units; b += NW) {
    Unit x;
    load(b, x);
    mul(x);
  }

#pragma unroll
  for (int j = 0; j < NF; ++j)
#pragma unroll
    for (int f = 0; f < MF; ++f) part[wave][j * MF + f][lane] = acc[j][f];
  __syncthreads();

  // A lane of fragment (j, f) holds row 16 f + l16 and, in register r, column 16 j + 4 q + r.
  auto finish = [&](auto ct) {
    constexpr int CT = decltype(ct)::value;
#pragma unroll
    for (int t = 0; t < MINE; ++t) {
      const int i = threadIdx.x + 64 * NW * t;
      int m, n;
      if (!item(i, m, n)) continue;
      float cin[4] = {};
      if (p.beta != 0.0f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) cin[e] = load_as_float<CT>(p.C, (int64_t)m * p.ldc + min(n + e, p.N - 1));
      }
      x_f32x4 v = x_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < NW; ++w) v += part[w][i >> 6][i & 63];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < p.N)
          store_from_float<CT>(p.C, (int64_t)m * p.ldc + n + e, epilogue_value<CT>(v[e], p.alpha, p.beta, cin[e], bj[t][e], p.epi));
    }
  };
  if (c_type == F32) finish(std::integral_constant<int, F32>{});
  else if (c_type == F16) finish(std::integral_constant<int, F16>{});
  else finish(std::integral_constant<int, BF16>{});
}

template <int NF, int MF, int U>
hipError_t launch_cfg(GemmParams p, GroupArgs ga, int c_type, hipStream_t s) {
  p.tiles_n = (p.N + 16 * NF - 1) / (16 * NF);
  const int64_t grid = whole_rounds(max_row_tiles(p.M, ga.groups, 16 * MF) * p.tiles_n);
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  return launch_in_slices(grid, 64 * NW, [&](int64_t first, unsigned n) {
    ga.first = (int)first;
    hipLaunchKernelGGL((mx_stream_kernel<NF, MF, U>), dim3(n), dim3(64 * NW), 0, s, p, ga, c_type);
  });
}

}  // namespace

// rows: 16, 32 or 64 rows of C per workgroup; columns: 16 (with 16 rows only) or 32.
hipError_t launch_stream_mx(const GemmParams& p, const GroupArgs& ga, int c_type, int rows, int columns, hipStream_t s) {
  if (columns == 16) {
    if (rows != 16) return hipErrorInvalidValue;
    // longer units where every wave has one (1 x 28672 x 8192 23.7 us against 26.9, 1 x 57344 x 2880 17.6 against 16.2)
    return p.K >= 6 * 64 * 8 ? launch_cfg<1, 1, 8>(p, ga, c_type, s) : launch_cfg<1, 1, 4>(p, ga, c_type, s);
  }
  switch (rows) {
    case 16: return launch_cfg<2, 1, 4>(p, ga, c_type, s);
    case 32: return launch_cfg<2, 2, 4>(p, ga, c_type, s);
    case 64: return launch_cfg<2, 4, 4>(p, ga, c_type, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tgemm
