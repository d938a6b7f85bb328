// Rows to the experts and back: A[place] = X[t], C[t] = sum of weight * Y[place], and the gradients.
//
// Everything goes by tokens: the places of a token's pairs are a few neighbouring numbers, a token's row
// is read (or written) once, and the experts' rows are whole rows, so that each 16-byte access of a wave
// lies in one run of 1 KB whatever the order.  What bounds it is the bytes.
#include <type_traits>

#include "experts.hpp"

namespace tgemm {

namespace {

typedef uint32_t m_u32x4 __attribute__((ext_vector_type(4)));

// Chunk c (16 bytes) of a row of K elements, zeros past its end; any alignment.
template <int ES>
__device__ __forceinline__ m_u32x4 load_chunk(const uint8_t* row, int64_t c, int K) {
  constexpr int CE = 16 / ES;
  m_u32x4 v = m_u32x4{0u, 0u, 0u, 0u};
  const int64_t k = c * CE;
  if (k + CE <= K) {
    __builtin_memcpy(&v, row + k * ES, 16);
  } else {
    for (int e = 0; e < CE; ++e)
      if (k + e < K) {
        if constexpr (ES == 4) v[e] = reinterpret_cast<const uint32_t*>(row)[k + e];
        else v[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[k + e] << (16 * (e & 1));
      }
  }
  return v;
}

template <int ES>
__device__ __forceinline__ void store_chunk(uint8_t* row, int64_t c, int K, m_u32x4 v) {
  constexpr int CE = 16 / ES;
  const int64_t k = c * CE;
  if (k + CE <= K) {
    __builtin_memcpy(row + k * ES, &v, 16);
  } else {
    for (int e = 0; e < CE; ++e)
      if (k + e < K) {
        if constexpr (ES == 4) reinterpret_cast<uint32_t*>(row)[k + e] = v[e];
        else reinterpret_cast<uint16_t*>(row)[k + e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
      }
  }
}

template <int DT>
__device__ __forceinline__ float element(m_u32x4 v, int e) {
  if constexpr (DT == F32) return __uint_as_float(v[e]);
  const uint32_t h = (v[e >> 1] >> (16 * (e & 1))) & 0xffffu;
  return DT == F16 ? f16_bits_to_float(h) : bf16_bits_to_float(h);
}

template <int DT>
__device__ __forceinline__ m_u32x4 pack(const float* f) {
  m_u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == F32) v[i] = __float_as_uint(f[i]);
    else if constexpr (DT == F16) v[i] = float_to_f16_bits(f[2 * i]) | float_to_f16_bits(f[2 * i + 1]) << 16;
    else v[i] = float_to_bf16_bits(f[2 * i]) | float_to_bf16_bits(f[2 * i + 1]) << 16;
  }
  return v;
}

// The work of dispatch and combine comes in pieces, 64 lanes x UNROLL chunks of one token's row, one to a
// wave.
constexpr int UNROLL = 4;
inline int64_t pieces(int64_t K, int es) { return (K * es + 64 * 16 * UNROLL - 1) / (64 * 16 * UNROLL); }

template <int ES>
__global__ __launch_bounds__(256) void dispatch_kernel(RowArgs p, int64_t first, int per) {
  const int lane = threadIdx.x & 63;
  const int64_t item = (first + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = item / per;
  if (t >= p.T) return;
  const int64_t c0 = (item - t * per) * (64 * UNROLL) + lane, chunks = ((int64_t)p.K * ES + 15) / 16;
  const uint8_t* const src = reinterpret_cast<const uint8_t*>(p.X) + t * p.ldx * ES;
  m_u32x4 v[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u)
    if (c0 + 64 * u < chunks) v[u] = load_chunk<ES>(src, c0 + 64 * u, p.K);
  for (int j = 0; j < p.top; ++j) {
    const int at = p.place[t * p.top + j];
    if (at < 0 || at >= p.R) continue;
    uint8_t* const dst = reinterpret_cast<uint8_t*>(p.Y) + at * p.ldy * ES;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (c0 + 64 * u < chunks) store_chunk<ES>(dst, c0 + 64 * u, p.K, v[u]);
  }
}

template <int DT>
__global__ __launch_bounds__(256) void combine_kernel(RowArgs p, int64_t first, int per) {
  constexpr int ES = DTypeInfo<DT>::bytes, CE = 16 / ES;
  const int lane = threadIdx.x & 63;
  const int64_t item = (first + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = item / per;
  if (t >= p.T) return;
  const int64_t c0 = (item - t * per) * (64 * UNROLL) + lane, chunks = ((int64_t)p.K * ES + 15) / 16;
  float sum[UNROLL][CE] = {};
  for (int j = 0; j < p.top; ++j) {
    const int at = p.place[t * p.top + j];
    if (at < 0 || at >= p.R) continue;
    const float w = p.weight ? p.weight[t * p.top + j] : 1.0f;
    const uint8_t* const src = reinterpret_cast<const uint8_t*>(p.X) + at * p.ldx * ES;
    m_u32x4 v[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (c0 + 64 * u < chunks) v[u] = load_chunk<ES>(src, c0 + 64 * u, p.K);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (c0 + 64 * u < chunks)
#pragma unroll
        for (int e = 0; e < CE; ++e) sum[u][e] = fmaf(w, element<DT>(v[u], e), sum[u][e]);
  }
  uint8_t* const dst = reinterpret_cast<uint8_t*>(p.Y) + t * p.ldy * ES;
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    if (c0 + 64 * u >= chunks) continue;
    if (p.beta != 0.0f) {
      const m_u32x4 c = load_chunk<ES>(dst, c0 + 64 * u, p.K);
#pragma unroll
      for (int e = 0; e < CE; ++e) sum[u][e] = fmaf(p.beta, element<DT>(c, e), sum[u][e]);
    }
    store_chunk<ES>(dst, c0 + 64 * u, p.K, pack<DT>(sum[u]));
  }
}

// The gradient of combine: TPR threads (a wave, four tokens a workgroup, or all 256) take one token, hold
// NV chunks of D each in registers and meet for the dot products, wave by wave in a fixed order.
template <int DT, int TPR, int NV>
__global__ __launch_bounds__(256) void combine_grad_kernel(RowGradArgs p, int64_t first) {
  constexpr int ES = DTypeInfo<DT>::bytes, CE = 16 / ES;
  __shared__ float part[4];
  const int tid = threadIdx.x, i = tid % TPR;
  const int64_t t = (first + blockIdx.x) * (256 / TPR) + tid / TPR;
  if (TPR == 64 && t >= p.T) return;
  const int64_t chunks = ((int64_t)p.K * ES + 15) / 16;
  const uint8_t* const D = reinterpret_cast<const uint8_t*>(p.D) + t * p.ldd * ES;
  m_u32x4 d[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u)
    if (i + u * TPR < chunks) d[u] = load_chunk<ES>(D, i + u * TPR, p.K);
  for (int j = 0; j < p.top; ++j) {
    const int64_t pair = t * p.top + j;
    const int at = p.place[pair];
    if (at < 0 || at >= p.R) {
      if (i == 0) p.dw[pair] = 0.0f;
      continue;
    }
    const float w = p.weight[pair];
    const uint8_t* const Y = reinterpret_cast<const uint8_t*>(p.Y) + at * p.ldy * ES;
    uint8_t* const dY = reinterpret_cast<uint8_t*>(p.dY) + at * p.lddy * ES;
    float dot = 0.0f;
    auto chunk = [&](int64_t c, m_u32x4 dv, m_u32x4 yv) {
      float o[CE];
#pragma unroll
      for (int e = 0; e < CE; ++e) {
        const float x = element<DT>(dv, e);
        dot = fmaf(x, element<DT>(yv, e), dot);
        o[e] = w * x;
      }
      store_chunk<ES>(dY, c, p.K, pack<DT>(o));
    };
    m_u32x4 y[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (i + u * TPR < chunks) y[u] = load_chunk<ES>(Y, i + u * TPR, p.K);
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (i + u * TPR < chunks) chunk(i + u * TPR, d[u], y[u]);
    for (int64_t c = i + NV * TPR; c < chunks; c += TPR) chunk(c, load_chunk<ES>(D, c, p.K), load_chunk<ES>(Y, c, p.K));
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) dot += __shfl_xor(dot, s);
    if constexpr (TPR > 64) {
      __syncthreads();
      if ((tid & 63) == 0) part[tid >> 6] = dot;
      __syncthreads();
      dot = (part[0] + part[1]) + (part[2] + part[3]);
    }
    if (i == 0) p.dw[pair] = dot;
  }
}

template <int DT, int TPR, int NV>
hipError_t grad_cfg(const RowGradArgs& p, hipStream_t s) {
  constexpr int RPW = 256 / TPR;
  return launch_in_slices(((int64_t)p.T + RPW - 1) / RPW, 256, [&](int64_t first, unsigned n) {
    hipLaunchKernelGGL((combine_grad_kernel<DT, TPR, NV>), dim3(n), dim3(256), 0, s, p, first);
  });
}

template <int DT>
hipError_t grad_type(const RowGradArgs& p, hipStream_t s) {
  const int64_t chunks = ((int64_t)p.K * DTypeInfo<DT>::bytes + 15) / 16;
  if (chunks <= 64 * 4) return grad_cfg<DT, 64, 4>(p, s);
  return grad_cfg<DT, 256, 4>(p, s);
}

}  // namespace

hipError_t launch_dispatch_rows(const RowArgs& p, int type, hipStream_t s) {
  const int64_t per = pieces(p.K, type == F32 ? 4 : 2);
  return launch_in_slices((p.T * per + 3) / 4, 256, [&](int64_t first, unsigned n) {
    if (type == F32) hipLaunchKernelGGL((dispatch_kernel<4>), dim3(n), dim3(256), 0, s, p, first, (int)per);
    else hipLaunchKernelGGL((dispatch_kernel<2>), dim3(n), dim3(256), 0, s, p, first, (int)per);
  });
}

hipError_t launch_combine_rows(const RowArgs& p, int type, hipStream_t s) {
  const int64_t per = pieces(p.K, type == F32 ? 4 : 2);
  return launch_in_slices((p.T * per + 3) / 4, 256, [&](int64_t first, unsigned n) {
    if (type == F32) hipLaunchKernelGGL((combine_kernel<F32>), dim3(n), dim3(256), 0, s, p, first, (int)per);
    else if (type == F16) hipLaunchKernelGGL((combine_kernel<F16>), dim3(n), dim3(256), 0, s, p, first, (int)per);
    else hipLaunchKernelGGL((combine_kernel<BF16>), dim3(n), dim3(256), 0, s, p, first, (int)per);
  });
}

hipError_t launch_combine_rows_grad(const RowGradArgs& p, int type, hipStream_t s) {
  return type == F32 ? grad_type<F32>(p, s) : type == F16 ? grad_type<F16>(p, s) : grad_type<BF16>(p, s);
}

}  // namespace tgemm
