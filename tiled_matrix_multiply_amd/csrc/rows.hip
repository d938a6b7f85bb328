// Rows to the experts and back: A[place] = X[t], C[t] = sum of weight * Y[place], and the gradients.
//
// Everything goes by tokens: the places of a token's pairs are a few neighbouring numbers, a token's row
// is read (or written) once, and the experts' rows are whole rows, so that each 16-byte access of a wave
// lies in one run of 1 KB whatever the order.  What bounds it is the bytes: 8190 tokens of 8 x 2048 in bf16
// dispatched in 58.8 us (5.13 TB/s), combined in 51.3 (5.88), the gradient 118.2 (4.82), where a copy of
// 4 GiB runs at 4.63.
#include <type_traits>

#include "experts.hpp"

namespace tgemm {

namespace {

typedef uint32_t m_u32x4 __attribute__((ext_vector_type(4)));
typedef m_u32x4 m_any4 __attribute__((aligned(2)));

// Chunk c (16 bytes) of a row of K elements, zeros past its end; any alignment.  NT: not kept in the caches.
template <int ES, bool NT = false>
__device__ __forceinline__ m_u32x4 load_chunk(const uint8_t* row, int64_t c, int K) {
  constexpr int CE = 16 / ES;
  m_u32x4 v = m_u32x4{0u, 0u, 0u, 0u};
  const int64_t k = c * CE;
  if (k + CE <= K) {
    if constexpr (NT) v = __builtin_nontemporal_load(reinterpret_cast<const m_any4*>(row + k * ES));
    else __builtin_memcpy(&v, row + k * ES, 16);
  } else {
    for (int e = 0; e < CE; ++e)
      if (k + e < K) {
        if constexpr (ES == 4) v[e] = reinterpret_cast<const uint32_t*>(row)[k + e];
        else v[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[k + e] << (16 * (e & 1));
      }
  }
  return v;
}

template <int ES, bool NT = false>
__device__ __forceinline__ void store_chunk(uint8_t* row, int64_t c, int K, m_u32x4 v) {
  constexpr int CE = 16 / ES;
  const int64_t k = c * CE;
  if (k + CE <= K) {
    if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<m_any4*>(row + k * ES));
    else __builtin_memcpy(row + k * ES, &v, 16);
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

// The work of dispatch and combine comes in pieces of 64 chunks of one token's row, one to a wave.  (Four
// chunks a lane, the loads together, were slower everywhere: fewer waves have more to wait for.  4096 tokens
// to 2 places of 4096: dispatch 16.1 us with one, 16.0 with two, 16.4 with four; combine 19.4, 21.1, 23.6;
// 512 tokens to 8: dispatch 7.5, 7.6, 8.7, combine 7.6, 9.1, 14.7.)
inline int64_t pieces(int64_t K, int es) { return (K * es + 64 * 16 - 1) / (64 * 16); }

// A wave's token and chunk.
struct Piece {
  int64_t t, c;
  __device__ __forceinline__ Piece(int64_t first, int per) {
    const int64_t item = (first + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    t = item / per;
    c = (item - t * per) * 64 + (threadIdx.x & 63);
  }
};

template <int ES, bool NT>
__global__ __launch_bounds__(256) void dispatch_kernel(RowArgs p, int64_t first, int per) {
  const Piece at(first, per);
  if (at.t >= p.T || at.c * (16 / ES) >= p.K) return;
  const m_u32x4 v = load_chunk<ES>(reinterpret_cast<const uint8_t*>(p.X) + at.t * p.ldx * ES, at.c, p.K);
  for (int j = 0; j < p.top; ++j) {
    const int row = p.place[at.t * p.top + j];
    if (row < 0 || row >= p.R) continue;
    store_chunk<ES, NT>(reinterpret_cast<uint8_t*>(p.Y) + row * p.ldy * ES, at.c, p.K, v);
  }
}

// Places of a token's J pairs from j on, which of them are rows at all, and their weights.  (A row that is
// none is read as row 0 and not used: loads outside branches go out together.)
template <int J>
struct Pairs {
  int at[J];
  bool ok[J];
  float w[J];
  __device__ __forceinline__ Pairs(const int32_t* place, const float* weight, int64_t first, int j, int top, int R) {
#pragma unroll
    for (int q = 0; q < J; ++q) {
      const int64_t pair = first + min(j + q, top - 1);
      const int row = place[pair];
      ok[q] = j + q < top && row >= 0 && row < R;
      at[q] = row >= 0 && row < R ? row : 0;
      w[q] = weight ? weight[pair] : 1.0f;
    }
  }
};

template <int DT, int J, bool NT>
__global__ __launch_bounds__(256) void combine_kernel(RowArgs p, int64_t first, int per) {
  constexpr int ES = DTypeInfo<DT>::bytes, CE = 16 / ES;
  const Piece at(first, per);
  if (at.t >= p.T || at.c * CE >= p.K) return;
  float sum[CE] = {};
  for (int j = 0; j < p.top && p.R > 0; j += J) {
    const Pairs<J> pairs(p.place, p.weight, at.t * p.top, j, p.top, p.R);
    m_u32x4 v[J];
#pragma unroll
    for (int q = 0; q < J; ++q)
      v[q] = load_chunk<ES, NT>(reinterpret_cast<const uint8_t*>(p.X) + pairs.at[q] * p.ldx * ES, at.c, p.K);
#pragma unroll
    for (int q = 0; q < J; ++q) {
      if (!pairs.ok[q]) continue;
#pragma unroll
      for (int e = 0; e < CE; ++e) sum[e] = fmaf(pairs.w[q], element<DT>(v[q], e), sum[e]);
    }
  }
  uint8_t* const dst = reinterpret_cast<uint8_t*>(p.Y) + at.t * p.ldy * ES;
  if (p.beta != 0.0f) {
    const m_u32x4 c = load_chunk<ES>(dst, at.c, p.K);
#pragma unroll
    for (int e = 0; e < CE; ++e) sum[e] = fmaf(p.beta, element<DT>(c, e), sum[e]);
  }
  store_chunk<ES, NT>(dst, at.c, p.K, pack<DT>(sum));
}

// The sum over a wave, in every lane, in a fixed order.
__device__ __forceinline__ float wave_sum(float v) {
  auto turn = [](float x, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  v += turn(v, std::integral_constant<int, 0x128>{});  // row_ror 8, 4, 2, 1
  v += turn(v, std::integral_constant<int, 0x124>{});
  v += turn(v, std::integral_constant<int, 0x122>{});
  v += turn(v, std::integral_constant<int, 0x121>{});
  auto of = [](float x, int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), l)); };
  return (of(v, 0) + of(v, 16)) + (of(v, 32) + of(v, 48));
}

// The gradient of combine: TPR threads (a wave, four tokens a workgroup, or all 256) take one token, hold
// NV chunks of D each in registers, take J rows together and meet for the dot products, wave by wave in
// a fixed order, for MEET pairs at a time.
template <int DT, int TPR, int NV, int J, bool NT>
__global__ __launch_bounds__(256) void combine_grad_kernel(RowGradArgs p, int64_t first) {
  constexpr int ES = DTypeInfo<DT>::bytes, CE = 16 / ES, MEET = 8;
  static_assert(MEET % J == 0, "whole batches");
  __shared__ float part[4][MEET];
  const int tid = threadIdx.x, i = tid % TPR;
  const int64_t t = (first + blockIdx.x) * (256 / TPR) + (TPR == 64 ? __builtin_amdgcn_readfirstlane(tid >> 6) : 0);
  if (TPR == 64 && t >= p.T) return;
  const int64_t chunks = ((int64_t)p.K * ES + 15) / 16;
  const uint8_t* const D = reinterpret_cast<const uint8_t*>(p.D) + t * p.ldd * ES;
  m_u32x4 d[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u)
    if (i + u * TPR < chunks) d[u] = load_chunk<ES, NT>(D, i + u * TPR, p.K);
  for (int j = 0; j < p.top; j += J) {
    const Pairs<J> pairs(p.place, p.weight, t * p.top, j, p.top, p.R);
    float dot[J] = {};
    auto chunk = [&](int q, int64_t c, m_u32x4 dv, m_u32x4 yv) {
      float o[CE];
#pragma unroll
      for (int e = 0; e < CE; ++e) {
        const float x = element<DT>(dv, e);
        dot[q] = fmaf(x, element<DT>(yv, e), dot[q]);
        o[e] = pairs.w[q] * x;
      }
      store_chunk<ES>(reinterpret_cast<uint8_t*>(p.dY) + pairs.at[q] * p.lddy * ES, c, p.K, pack<DT>(o));
    };
    if (p.R > 0) {
      m_u32x4 y[J][NV];
#pragma unroll
      for (int q = 0; q < J; ++q)
#pragma unroll
        for (int u = 0; u < NV; ++u)
          if (i + u * TPR < chunks)
            y[q][u] =
                load_chunk<ES, NT>(reinterpret_cast<const uint8_t*>(p.Y) + pairs.at[q] * p.ldy * ES, i + u * TPR, p.K);
#pragma unroll
      for (int q = 0; q < J; ++q) {
        if (!pairs.ok[q]) continue;
#pragma unroll
        for (int u = 0; u < NV; ++u)
          if (i + u * TPR < chunks) chunk(q, i + u * TPR, d[u], y[q][u]);
        const uint8_t* const Y = reinterpret_cast<const uint8_t*>(p.Y) + pairs.at[q] * p.ldy * ES;
        for (int64_t c = i + NV * TPR; c < chunks; c += TPR) chunk(q, c, load_chunk<ES>(D, c, p.K), load_chunk<ES>(Y, c, p.K));
      }
    }
#pragma unroll
    for (int q = 0; q < J; ++q) {
      const float s = wave_sum(dot[q]);
      if constexpr (TPR == 64) {
        if (i == 0 && j + q < p.top) p.dw[t * p.top + j + q] = s;
      } else if ((tid & 63) == 0) {
        part[tid >> 6][(j + q) % MEET] = s;
      }
    }
    if constexpr (TPR > 64) {
      if ((j + J) % MEET == 0 || j + J >= p.top) {
        __syncthreads();
        const int from = j / MEET * MEET;
        if (tid < MEET && from + tid < p.top)
          p.dw[t * p.top + from + tid] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
        __syncthreads();
      }
    }
  }
}

// What the caches are not to keep.  The memory-side cache holds 256 MB, and a call's rows push out of it what
// the next call could have read there: rows that are read for the last time (combine and its gradient) and
// the sums of many go past it.  8190 tokens dispatched to 8 rows of 2048 and others combined: 139.5 us with
// ordinary accesses, 108.3 so; 4096 to 2 of 4096, both ways with all gradients: 85.5 and 83.6, 16384 to 2: 372
// and 324; but 512 to 8 of 4096, 34 MB of rows, which stay there from call to call: 37.4 and 40.6.  Dispatched
// rows are read next, so they go past it only where it could not hold them (16384 to 2 of 4096, 268 MB,
// dispatched and others combined: 143.9 us with ordinary stores, 125.9 so, and the same for the same rows; 8190 to
// 8 of 2048, the same rows combined: 90.7 and 103.8).
inline bool past_caches(int64_t T, int64_t top, int64_t K, int es, int64_t bytes) {
  return (__int128)(T * top) * K * es >= bytes;
}
constexpr int64_t kReadOnce = int64_t(48) << 20, kTooLarge = int64_t(256) << 20;

template <int DT, int TPR, int NV, int J>
hipError_t grad_cfg(const RowGradArgs& p, hipStream_t s) {
  constexpr int RPW = 256 / TPR;
  const bool nt = past_caches(p.T, p.top, p.K, DTypeInfo<DT>::bytes, kReadOnce);
  return launch_in_slices(((int64_t)p.T + RPW - 1) / RPW, 256, [&](int64_t first, unsigned n) {
    if (nt) hipLaunchKernelGGL((combine_grad_kernel<DT, TPR, NV, J, true>), dim3(n), dim3(256), 0, s, p, first);
    else hipLaunchKernelGGL((combine_grad_kernel<DT, TPR, NV, J, false>), dim3(n), dim3(256), 0, s, p, first);
  });
}

// A wave is enough for a row of 2 KB and spares the meeting (8192 tokens of 4 x 1024: 33.2 us against 46.2,
// 16384 of 8 x 512: 61.8 against 127.4); of longer rows a wave takes too long over one token (8190 of 8 x
// 2048: 129.2 against 117.5; 512 of 8 x 4096: 34.4 against 13.5).  Two chunks a thread, four where the row has
// them (4096 of 8 x 7168: 205 us against 216).  Two pairs together, unless there is one alone (8192 of 1 x
// 4096: 34.0 us against 38.5 with a second that is none).
template <int DT, int J>
hipError_t grad_pairs(const RowGradArgs& p, hipStream_t s) {
  const int64_t chunks = ((int64_t)p.K * DTypeInfo<DT>::bytes + 15) / 16;
  if (chunks <= 64 * 2) return grad_cfg<DT, 64, 2, J>(p, s);
  if (chunks <= 256 * 2) return grad_cfg<DT, 256, 2, J>(p, s);
  return grad_cfg<DT, 256, 4, J>(p, s);
}
template <int DT>
hipError_t grad_type(const RowGradArgs& p, hipStream_t s) {
  return p.top == 1 ? grad_pairs<DT, 1>(p, s) : grad_pairs<DT, 2>(p, s);
}

// Two pairs together as well (8192 tokens of 1 x 4096: 27.0 us with one, 30.2 with two; 4096 of 2 x 4096: 20.3
// and 19.4; more gain nothing for 8 pairs and cost for fewer).
template <int DT, int J>
hipError_t combine_cfg(const RowArgs& p, hipStream_t s) {
  const int64_t per = pieces(p.K, DTypeInfo<DT>::bytes);
  const bool nt = past_caches(p.T, p.top, p.K, DTypeInfo<DT>::bytes, kReadOnce);
  return launch_in_slices((p.T * per + 3) / 4, 256, [&](int64_t first, unsigned n) {
    if (nt) hipLaunchKernelGGL((combine_kernel<DT, J, true>), dim3(n), dim3(256), 0, s, p, first, (int)per);
    else hipLaunchKernelGGL((combine_kernel<DT, J, false>), dim3(n), dim3(256), 0, s, p, first, (int)per);
  });
}
template <int DT>
hipError_t combine_type(const RowArgs& p, hipStream_t s) {
  return p.top == 1 ? combine_cfg<DT, 1>(p, s) : combine_cfg<DT, 2>(p, s);
}

template <int ES, bool NT>
hipError_t dispatch_cfg(const RowArgs& p, hipStream_t s) {
  const int64_t per = pieces(p.K, ES);
  return launch_in_slices((p.T * per + 3) / 4, 256, [&](int64_t first, unsigned n) {
    hipLaunchKernelGGL((dispatch_kernel<ES, NT>), dim3(n), dim3(256), 0, s, p, first, (int)per);
  });
}

}  // namespace

hipError_t launch_dispatch_rows(const RowArgs& p, int type, hipStream_t s) {
  const int es = type == F32 ? 4 : 2;
  return past_caches(p.T, p.top, p.K, es, kTooLarge) ? (es == 4 ? dispatch_cfg<4, true>(p, s) : dispatch_cfg<2, true>(p, s))
                                                     : (es == 4 ? dispatch_cfg<4, false>(p, s) : dispatch_cfg<2, false>(p, s));
}

hipError_t launch_combine_rows(const RowArgs& p, int type, hipStream_t s) {
  return type == F32 ? combine_type<F32>(p, s) : type == F16 ? combine_type<F16>(p, s) : combine_type<BF16>(p, s);
}

hipError_t launch_combine_rows_grad(const RowGradArgs& p, int type, hipStream_t s) {
  return type == F32 ? grad_type<F32>(p, s) : type == F16 ? grad_type<F16>(p, s) : grad_type<BF16>(p, s);
}

}  // namespace tgemm
