// Grouped and 8-bit integer products for few rows per group (gfx950 only): decoding, where the
// weights are read once and nothing else matters.
//
// A workgroup owns a block of columns of one group and up to 16 MF of its rows; its waves share
// out K and meet in LDS at the end, in wave order.  Weights and rows go straight from global
// memory into the registers of 16 x 16 matrix instructions: nothing in the loop waits on another
// wave, and each wave keeps two sets of U steps (64 bytes of K) in flight.
//  * B stored N x K: a lane loads 16 bytes of K of its column, NF = 2 fragments of 16 columns.
//  * B stored K x N: a lane loads its 4 columns from each of the rows of K that its 16 bytes of a
//    fragment stand for and transposes them with byte permutes: 64 columns, NF = 4 fragments
//    (column 4 i + j of the block is row i of fragment j).
// What bounds it is the weights' bytes: 1 x 28672 x 8192 in 8 bits 46 us (5.1 TB/s), 32 rows over 64
// groups (23 of them with rows) of 1024 x 2048 19 us in bf16 (5.0 to 5.2 TB/s) and 11 us in 8 bits
// (4.5).  More than 64 groups cost each workgroup a walk over the offsets: 64 rows, one to a group, over
// 64, 128 and 256 groups 52, 51 and 55 us in bf16 and 31, 34 and 37 in 8 bits.
// With few columns it is the loads of a compute unit: 37 x 4104 x 4112 in 8 bits, stored K x N in
// 4-byte pieces, 12 us (1.4 TB/s).
// Any alignment and size: loads are unaligned, columns past N repeat the last ones and are not
// stored, and the last, partial step of K is loaded element by element.
#pragma once

#include <type_traits>

#include "grouped.hpp"

namespace tgemm {

typedef int s_i32x4 __attribute__((ext_vector_type(4)));
typedef float s_f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 s_bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 s_f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t s_u32x4 __attribute__((ext_vector_type(4)));

template <int DT, class Acc>
__device__ __forceinline__ Acc mma16(s_u32x4 x, s_u32x4 y, Acc c) {
  if constexpr (DT == I8)
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(s_i32x4, x), __builtin_bit_cast(s_i32x4, y), c, 0, 0, 0);
  else if constexpr (DT == BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(s_bf16x8, x), __builtin_bit_cast(s_bf16x8, y), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(s_f16x8, x), __builtin_bit_cast(s_f16x8, y), c, 0, 0, 0);
}

template <int DT, bool KN, int MF>
struct StreamCfg {
  static constexpr int ES = DTypeInfo<DT>::bytes, CE = 16 / ES;  // elements of a lane's 16 bytes
  static constexpr int KS = 64 / ES;                             // K of a step
  static constexpr int NF = KN ? 4 : 2, BN = 16 * NF, BM = 16 * MF;
  static constexpr int U = MF == 4 ? 2 : KN ? 2 : 4;             // steps loaded together
  static constexpr int CB = 4 * ES;                              // bytes of a K x N row a lane loads
  static constexpr int BD = KN ? CE * CB / 4 : 4 * NF;           // dwords of B a lane loads a step
  static constexpr int PART = NF * MF * 64 * 16;                 // bytes of one wave's sums
};

template <int DT, bool KN, int MF>
__global__ __launch_bounds__(MF == 1 ? 1024 : 512) void stream_kernel(GemmParams p, GroupArgs ga, int c_type) {
  using C = StreamCfg<DT, KN, MF>;
  using Acc = typename std::conditional<DT == I8, s_i32x4, s_f32x4>::type;
  constexpr int ES = C::ES, CE = C::CE, KS = C::KS, NF = C::NF, U = C::U;
  extern __shared__ __attribute__((aligned(16))) uint8_t part[];
  const int lane = threadIdx.x & 63, NW = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const GroupItem it = group_item(ga, p.M, C::BM, p.tiles_n, workgroup(ga), lane);
  if (it.group < 0) return;
  {
    const int ces = c_type == F32 ? 4 : 2;
    if (ces == 4) enter_group<ES, 4>(p, ga, it.group, it.row0, it.rows);
    else enter_group<ES, 2>(p, ga, it.group, it.row0, it.rows);
  }
  // the row tiles of a block of columns are neighbours: they share its weights in the L2
  const int tiles_m = (p.M + C::BM - 1) / C::BM;
  const int m0 = it.local % tiles_m * C::BM, n0 = it.local / tiles_m * C::BN;
  const int q = lane >> 4, l16 = lane & 15;

  const uint8_t* const A = reinterpret_cast<const uint8_t*>(p.A);
  const uint8_t* const B = reinterpret_cast<const uint8_t*>(p.B);
  // Lane offsets (32 bits: the host keeps a row under 2^23 bytes) from a uniform base.
  uint32_t oa[MF], ob[KN ? 1 : NF];
#pragma unroll
  for (int f = 0; f < MF; ++f) oa[f] = (uint32_t)((16 * f + l16 < p.M - m0 ? 16 * f + l16 : p.M - 1 - m0) * (int)(p.lda * ES)) + 16 * q;
  const uint8_t* const Ab = A + (int64_t)m0 * p.lda * ES;
  const int nc = n0 + 4 * l16;                      // K x N: the lane's columns, from nl on
  const int nl = KN ? min(nc, p.N - 4) : 0;
  const uint8_t* const Bb = KN ? B : B + (int64_t)n0 * p.ldb * ES;
  if constexpr (KN) {
    ob[0] = (uint32_t)(q * CE) * (uint32_t)(p.ldb * ES) + (uint32_t)nl * ES;
  } else {
#pragma unroll
    for (int f = 0; f < NF; ++f)
      ob[f] = (uint32_t)min(16 * f + l16, p.N - 1 - n0) * (uint32_t)(p.ldb * ES) + 16 * q;
  }

  struct Step {
    uint32_t b[C::BD];
    s_u32x4 a[MF];
  };
  auto load = [&](int s, Step& t) {
    const uint8_t* const as = Ab + (int64_t)s * 64;
#pragma unroll
    for (int f = 0; f < MF; ++f) __builtin_memcpy(&t.a[f], as + oa[f], 16);
    if constexpr (KN) {
      const int64_t row = p.ldb * ES;
      const uint8_t* const bs = Bb + (int64_t)s * KS * row;
#pragma unroll
      for (int i = 0; i < CE; ++i) __builtin_memcpy(&t.b[i * (C::CB / 4)], bs + i * row + ob[0], C::CB);
    } else {
      const uint8_t* const bs = Bb + (int64_t)s * 64;
#pragma unroll
      for (int f = 0; f < NF; ++f) __builtin_memcpy(&t.b[4 * f], bs + ob[f], 16);
    }
  };
  // The partial step after the last whole one: zeros past K on both sides.  A lane's 16 bytes are
  // whole, empty or, in at most one of the four quarters of the wave, cut.
  auto load_tail = [&](int s, Step& t) {
    const int64_t k = (int64_t)s * KS + q * CE;
    const int n = (int)min((int64_t)CE, max((int64_t)0, p.K - k));  // elements of this lane
    auto chunk = [&](const uint8_t* src) {
      s_u32x4 v = s_u32x4{0u, 0u, 0u, 0u};
      if (n == CE) {
        __builtin_memcpy(&v, src, 16);
      } else if (n > 0) {
        uint32_t x[CE];  // all loads first: past the end the last element once more
#pragma unroll
        for (int e = 0; e < CE; ++e) {
          const int at = min(e, n - 1);
          x[e] = ES == 1 ? src[at] : reinterpret_cast<const uint16_t*>(src)[at];
        }
#pragma unroll
        for (int e = 0; e < CE; ++e) v[e * ES / 4] |= (e < n ? x[e] : 0u) << (8 * (e * ES % 4));
      }
      return v;
    };
#pragma unroll
    for (int f = 0; f < MF; ++f) t.a[f] = chunk(Ab + (int64_t)s * 64 + oa[f]);
    if constexpr (KN) {
      const int64_t row = p.ldb * ES;
      const uint8_t* const bs = Bb + (int64_t)s * KS * row + nl * ES;
#pragma unroll
      for (int i = 0; i < CE; ++i) {  // past the end the matrix's last row once more
        const int64_t kr = min((int64_t)q * CE + i, (int64_t)p.K - 1 - (int64_t)s * KS);
        __builtin_memcpy(&t.b[i * (C::CB / 4)], bs + kr * row, C::CB);
      }
#pragma unroll
      for (int i = 0; i < CE; ++i)
#pragma unroll
        for (int d = 0; d < C::CB / 4; ++d)
          if (i >= n) t.b[i * (C::CB / 4) + d] = 0u;
    } else {
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const s_u32x4 v = chunk(Bb + (int64_t)s * 64 + ob[f]);
#pragma unroll
        for (int e = 0; e < 4; ++e) t.b[4 * f + e] = v[e];
      }
    }
  };
  // Fragment j of B from a step's registers.
  auto frags = [&](const Step& t, s_u32x4 (&b)[NF]) {
    if constexpr (!KN) {
#pragma unroll
      for (int f = 0; f < NF; ++f) b[f] = s_u32x4{t.b[4 * f], t.b[4 * f + 1], t.b[4 * f + 2], t.b[4 * f + 3]};
    } else if constexpr (ES == 2) {
      // row i of K holds columns 0, 1 in its first dword and 2, 3 in its second
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int d = 0; d < 4; ++d)
          b[j][d] = __builtin_amdgcn_perm(t.b[2 * (2 * d + 1) + j / 2], t.b[2 * (2 * d) + j / 2],
                                          j & 1 ? 0x07060302u : 0x05040100u);
    } else {
      // 4 x 4 bytes: rows 4 d .. 4 d + 3 of K, columns 0 .. 3
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t* r = &t.b[4 * d];
        const uint32_t x0 = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u), x1 = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u);
        const uint32_t y0 = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u), y1 = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
        b[0][d] = __builtin_amdgcn_perm(x1, x0, 0x05040100u);
        b[1][d] = __builtin_amdgcn_perm(x1, x0, 0x07060302u);
        b[2][d] = __builtin_amdgcn_perm(y1, y0, 0x05040100u);
        b[3][d] = __builtin_amdgcn_perm(y1, y0, 0x07060302u);
      }
    }
  };
  Acc acc[NF][MF];
#pragma unroll
  for (int j = 0; j < NF; ++j)
#pragma unroll
    for (int f = 0; f < MF; ++f) acc[j][f] = Acc{0, 0, 0, 0};
  auto mul = [&](const Step& t) {
    s_u32x4 b[NF];
    frags(t, b);
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int f = 0; f < MF; ++f) acc[j][f] = mma16<DT>(b[j], t.a[f], acc[j][f]);
  };

  // Whole steps in blocks of U, block after block over the waves; the last few steps and the
  // partial one go to one wave each, before its blocks.  Every load of the loop is unconditional
  // and its place among the loads in flight known at compile time: a load inside a branch would
  // make every wait behind it wait for all of them.
  const int steps = p.K / KS, blocks = steps / U, rest = steps - blocks * U;
  Step x[U], y[U];
  auto load_block = [&](int b, Step (&t)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) load(b * U + u, t[u]);
  };
  auto mul_block = [&](const Step (&t)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) mul(t[u]);
  };
  if (wave < rest) {
    load(blocks * U + wave, y[0]);
    mul(y[0]);
  } else if (wave == rest && steps * KS < p.K) {
    load_tail(steps, y[0]);
    mul(y[0]);
  }
  if (wave < blocks) {
    int b = wave;
    load_block(b, x);
    for (; b + 2 * NW < blocks; b += 2 * NW) {
      load_block(b + NW, y);
      mul_block(x);
      load_block(b + 2 * NW, x);
      mul_block(y);
    }
    if (b + NW < blocks) {
      load_block(b + NW, y);
      mul_block(x);
      mul_block(y);
    } else {
      mul_block(x);
    }
  }

  Acc* const mine = reinterpret_cast<Acc*>(part + wave * C::PART);
#pragma unroll
  for (int j = 0; j < NF; ++j)
#pragma unroll
    for (int f = 0; f < MF; ++f) mine[(j * MF + f) * 64 + lane] = acc[j][f];
  __syncthreads();

  // Item i of 16 MF rows x BN columns in runs of four columns.  A lane of fragment (j, f) holds row
  // 16 f + l16 and, in register r, the fragment's row 4 q + r.
  auto finish = [&](auto ct) {
    constexpr int CT = decltype(ct)::value;
    for (int i = threadIdx.x; i < NF * MF * 64; i += blockDim.x) {
      int m, n;
      const int r = i & 3, l = KN ? (i >> 2) & 63 : i & 63, jf = KN ? i >> 8 : i >> 6;
      if constexpr (KN) {
        m = m0 + 16 * jf + (l & 15);
        n = n0 + 16 * (l >> 4) + 4 * r;
      } else {
        m = m0 + 16 * (jf % MF) + (l & 15);
        n = n0 + 16 * (jf / MF) + 4 * (l >> 4);
      }
      if (m >= p.M || n >= p.N) continue;
      // K x N: where the lane's columns were moved back from the edge, column e of them is base + e
      const int base = KN ? min(n, p.N - 4) : n;
      // all reads together, past the edge the last column once more
      float bj[4], rb[4], cin[4];
      const float ra = DT == I8 ? p.alpha * p.ra[m] : p.alpha;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = min(base + e, p.N - 1);
        bj[e] = (p.epi & EPI_BIAS) ? p.bias[col] : 0.0f;
        rb[e] = DT == I8 ? p.rb[col] : 1.0f;
        cin[e] = p.beta != 0.0f ? load_as_float<CT>(p.C, (int64_t)m * p.ldc + col) : 0.0f;
      }
      Acc v = Acc{0, 0, 0, 0};
      for (int w = 0; w < NW; ++w) {
        const Acc* src = reinterpret_cast<const Acc*>(part + w * C::PART);
        if constexpr (KN) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] += src[(j * MF + jf) * 64 + l][r];
        } else {
          v += src[jf * 64 + l];
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float s = DT == I8 ? ((float)v[e] * ra) * rb[e] : (float)v[e];
        const float out = epilogue_value<CT>(s, DT == I8 ? 1.0f : ra, p.beta, cin[e], bj[e], p.epi);
        if (base + e >= n && base + e < p.N) store_from_float<CT>(p.C, (int64_t)m * p.ldc + base + e, out);
      }
    }
  };
  if constexpr (DT == I8) {
    if (c_type == F32) finish(std::integral_constant<int, F32>{});
    else if (c_type == F16) finish(std::integral_constant<int, F16>{});
    else finish(std::integral_constant<int, BF16>{});
  } else {
    finish(std::integral_constant<int, DT>{});
  }
}

template <int DT, bool KN, int MF>
hipError_t launch_stream_cfg(GemmParams p, GroupArgs ga, int c_type, int waves, hipStream_t s) {
  using C = StreamCfg<DT, KN, MF>;
  p.tiles_n = (p.N + C::BN - 1) / C::BN;
  const int64_t grid = whole_rounds(max_row_tiles(p.M, ga.groups, C::BM) * p.tiles_n);
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  return launch_in_slices(grid, 64 * waves, [&](int64_t first, unsigned n) {
    ga.first = (int)first;
    hipLaunchKernelGGL((stream_kernel<DT, KN, MF>), dim3(n), dim3(64 * waves), waves * C::PART, s, p, ga, c_type);
  });
}

// rows: 16, 32 or 64 rows of C per workgroup.
template <int DT>
hipError_t launch_stream_type(const GemmParams& p, const GroupArgs& ga, int c_type, bool kn, int rows, int waves,
                              hipStream_t s) {
  switch (rows * 2 + kn) {
    case 32: return launch_stream_cfg<DT, false, 1>(p, ga, c_type, waves, s);
    case 33: return launch_stream_cfg<DT, true, 1>(p, ga, c_type, waves, s);
    case 64: return launch_stream_cfg<DT, false, 2>(p, ga, c_type, waves, s);
    case 65: return launch_stream_cfg<DT, true, 2>(p, ga, c_type, waves, s);
    case 128: return launch_stream_cfg<DT, false, 4>(p, ga, c_type, waves, s);
    case 129: return launch_stream_cfg<DT, true, 4>(p, ga, c_type, waves, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tgemm
