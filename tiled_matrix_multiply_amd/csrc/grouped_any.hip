// Grouped and 8-bit integer products at any alignment, layout and size.
//
// The simplest kernel that is right for every case: 256 threads own a 64 x 64 tile of a group's
// C; every K slice of 64 bytes is read element by element (so no row needs an alignment), with
// zeros past the edges, through registers into LDS rows padded to 80 bytes (eight consecutive
// rows start on different banks); each of the four waves multiplies a 32 x 32 quarter on the
// matrix cores.  What bounds it is the element loads: one address per element.  The tiled
// kernels take over wherever rows start on 16 bytes.
#include <type_traits>

#include "grouped.hpp"

namespace tgemm {

namespace {

typedef float f32x16a __attribute__((ext_vector_type(16)));
typedef int i32x16a __attribute__((ext_vector_type(16)));
typedef int i32x4a __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8a __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8a __attribute__((ext_vector_type(8)));

constexpr int kT = 64, kRow = 80, kSliceBytes = 64;

template <int DT, class Acc>
__device__ __forceinline__ Acc mma_any(i32x4a x, i32x4a y, Acc c) {
  if constexpr (DT == I8) return __builtin_amdgcn_mfma_i32_32x32x32_i8(x, y, c, 0, 0, 0);
  else if constexpr (DT == BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8a, x), __builtin_bit_cast(bf16x8a, y), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8a, x), __builtin_bit_cast(f16x8a, y), c, 0, 0, 0);
}

// WG: the weight gradient (the sum runs over a group's rows).  a_mn / b_mn: A stored K x M, B
// stored K x N (the contiguous direction is M or N).
template <int DT, int CT, bool WG>
__global__ __launch_bounds__(256) void any_kernel(GemmParams p, GroupArgs ga, int a_mn, int b_mn) {
  using E = typename std::conditional<DT == I8, uint8_t, uint16_t>::type;
  using Acc = typename std::conditional<DT == I8, i32x16a, f32x16a>::type;
  constexpr int ES = sizeof(E), KS = kSliceBytes / ES, NE = kT * KS / 256;
  __shared__ __attribute__((aligned(16))) uint8_t As[2][kT * kRow], Bs[2][kT * kRow];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;

  int local;
  if constexpr (WG) {
    const int per = p.tiles_m * p.tiles_n, g = (int)(blockIdx.x / per);
    local = (int)(blockIdx.x % per);
    const GroupLane r = group_rows(ga, p.K, g, lane);
    enter_group_wgrad<ES, DTypeInfo<CT>::bytes>(p, ga, g, r.row0, r.rows);
  } else {
    const GroupItem it = group_item(ga, p.M, kT, p.tiles_n, (int)blockIdx.x, lane);
    if (it.group < 0) return;
    local = it.local;
    enter_group<ES, DTypeInfo<CT>::bytes>(p, ga, it.group, it.row0, it.rows);
  }
  const int m0 = local / p.tiles_n * kT, n0 = local % p.tiles_n * kT;
  const E* const A = reinterpret_cast<const E*>(p.A);
  const E* const B = reinterpret_cast<const E*>(p.B);

  // Element q of this thread's share of a slice, so that neighbouring lanes read neighbouring
  // addresses: along k, or along m / n.
  auto place = [&](int q, int mn, int& x, int& k) {
    const int e = tid + 256 * q;
    if (mn) { x = e & (kT - 1); k = e / kT; }
    else    { x = e / KS; k = e % KS; }
  };
  E ra[NE], rb[NE];
  auto fetch = [&](int s) {
#pragma unroll
    for (int q = 0; q < NE; ++q) {
      int x, k;
      place(q, a_mn, x, k);
      int64_t gx = m0 + x, gk = (int64_t)s * KS + k;
      ra[q] = gx < p.M && gk < p.K ? A[a_mn ? gk * p.lda + gx : gx * p.lda + gk] : (E)0;
      place(q, b_mn, x, k);
      gx = n0 + x;
      gk = (int64_t)s * KS + k;
      rb[q] = gx < p.N && gk < p.K ? B[b_mn ? gk * p.ldb + gx : gx * p.ldb + gk] : (E)0;
    }
  };
  auto stash = [&](int buf) {
#pragma unroll
    for (int q = 0; q < NE; ++q) {
      int x, k;
      place(q, a_mn, x, k);
      *reinterpret_cast<E*>(As[buf] + x * kRow + k * ES) = ra[q];
      place(q, b_mn, x, k);
      *reinterpret_cast<E*>(Bs[buf] + x * kRow + k * ES) = rb[q];
    }
  };

  Acc acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32, lrow = lane & 31, half = lane >> 5;
  const int slices = (int)(((int64_t)p.K + KS - 1) / KS);
  if (slices > 0) {
    fetch(0);
    stash(0);
    __syncthreads();
  }
  for (int s = 0; s < slices; ++s) {
    const int buf = s & 1;
    if (s + 1 < slices) fetch(s + 1);
#pragma unroll
    for (int g = 0; g < 2; ++g) {  // 32 bytes of k a step, 16 for each half of the lanes
      const i32x4a a = *reinterpret_cast<const i32x4a*>(As[buf] + (wm + lrow) * kRow + 32 * g + 16 * half);
      const i32x4a b = *reinterpret_cast<const i32x4a*>(Bs[buf] + (wn + lrow) * kRow + 32 * g + 16 * half);
      acc = mma_any<DT>(b, a, acc);
    }
    if (s + 1 < slices) stash(buf ^ 1);
    __syncthreads();
  }

  // The lane holds column lrow of D, a row of C, and in register r its column 8 (r / 4) + 4 half
  // + r % 4.
  const int m = m0 + wm + lrow;
  if (m >= p.M) return;
  const float sa = DT == I8 ? p.alpha * p.ra[m] : 1.0f;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int n = n0 + wn + 8 * (r >> 2) + 4 * half + (r & 3);
    if (n >= p.N) continue;
    const int64_t idx = (int64_t)m * p.ldc + n;
    const float cin = p.beta != 0.0f ? load_as_float<CT>(p.C, idx) : 0.0f;
    const float bj = (p.epi & EPI_BIAS) ? p.bias[n] : 0.0f;
    float v, scale;
    if constexpr (DT == I8) {
      v = ((float)acc[r] * sa) * p.rb[n];
      scale = 1.0f;
    } else {
      v = acc[r];
      scale = p.alpha;
    }
    store_from_float<CT>(p.C, idx, epilogue_value<CT>(v, scale, p.beta, cin, bj, p.epi));
  }
}

// dbias_g[n] = the sum of D's rows of group g: 64 columns a workgroup, its four waves take every
// fourth row and meet in LDS (the order of the sum depends on the group's size alone).
template <int DT>
__global__ __launch_bounds__(256) void bias_grad_kernel(const uint16_t* D, int64_t ldd, int M, int N,
                                                        GroupArgs ga, float* dbias) {
  __shared__ float part[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = blockIdx.y;
  const GroupLane r = group_rows(ga, M, g, lane);
  const int n = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (n < N)
    for (int i = wave; i < r.rows; i += 4)
      s += load_as_float<DT>(D, ((int64_t)r.row0 + i) * ldd + n);
  part[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && n < N) dbias[(int64_t)g * N + n] = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
}

template <int DT, int CT, bool WG>
hipError_t launch_any_cfg(GemmParams p, const GroupArgs& ga, bool a_mn, bool b_mn, hipStream_t s) {
  p.tiles_m = (p.M + kT - 1) / kT;
  p.tiles_n = (p.N + kT - 1) / kT;
  const int64_t rows = WG ? (int64_t)p.tiles_m * ga.groups : max_row_tiles(p.M, ga.groups, kT);
  const int64_t grid = rows * p.tiles_n;
  if (grid <= 0) return hipSuccess;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((any_kernel<DT, CT, WG>), dim3((unsigned)grid), dim3(256), 0, s, p, ga, (int)a_mn, (int)b_mn);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_any(const GemmParams& p, const GroupArgs& ga, int type, int c_type, bool b_mn,
                              hipStream_t s) {
  switch (type * 16 + c_type) {
    case F16 * 16 + F16: return launch_any_cfg<F16, F16, false>(p, ga, false, b_mn, s);
    case BF16 * 16 + BF16: return launch_any_cfg<BF16, BF16, false>(p, ga, false, b_mn, s);
    case I8 * 16 + F16: return launch_any_cfg<I8, F16, false>(p, ga, false, b_mn, s);
    case I8 * 16 + BF16: return launch_any_cfg<I8, BF16, false>(p, ga, false, b_mn, s);
    case I8 * 16 + F32: return launch_any_cfg<I8, F32, false>(p, ga, false, b_mn, s);
    default: return hipErrorInvalidValue;
  }
}

// p.M x p.N: the gradient as stored; p.A and p.B: the rows it is the product of; p.K: all rows.
hipError_t launch_grouped_wgrad_any(const GemmParams& p, const GroupArgs& ga, int type, int c_type,
                                    hipStream_t s) {
  switch (type * 16 + c_type) {
    case F16 * 16 + F16: return launch_any_cfg<F16, F16, true>(p, ga, true, true, s);
    case BF16 * 16 + BF16: return launch_any_cfg<BF16, BF16, true>(p, ga, true, true, s);
    case F16 * 16 + F32: return launch_any_cfg<F16, F32, true>(p, ga, true, true, s);
    case BF16 * 16 + F32: return launch_any_cfg<BF16, F32, true>(p, ga, true, true, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_bias_grad(const void* D, int64_t ldd, int M, int N, int type, const GroupArgs& ga,
                            float* dbias, hipStream_t s) {
  if (N <= 0 || ga.groups <= 0) return hipSuccess;
  const dim3 grid((unsigned)((N + 63) / 64), (unsigned)ga.groups);
  const uint16_t* d = reinterpret_cast<const uint16_t*>(D);
  if (type == F16) hipLaunchKernelGGL((bias_grad_kernel<F16>), grid, dim3(256), 0, s, d, ldd, M, N, ga, dbias);
  else hipLaunchKernelGGL((bias_grad_kernel<BF16>), grid, dim3(256), 0, s, d, ldd, M, N, ga, dbias);
  return hipGetLastError();
}

}  // namespace tgemm
