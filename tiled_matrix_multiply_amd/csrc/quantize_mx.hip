// Rows in MXFP4: for every 32 elements a power of two and 4-bit elements (E2M1).
//
// A lane takes 8 neighbouring elements, four lanes a block: the largest magnitude meets in two steps
// across the four, and each lane's 8 codes are 4 bytes, so that a wave stores 256 bytes of codes and 16
// of scales together.  The conversion instruction divides by the power of two, rounds to nearest, ties
// to even, and saturates (all 16-bit values against the definition: tests).  What bounds it is the bytes: bf16,
// 16384 x 4096 29.7 us (5.7 TB/s), 4096 x 4096 8.6 (4.9), 8190 x 2048 to 8 places each 19.1 (5.5).
#include "experts.hpp"

namespace tgemm {

namespace {

typedef uint32_t z_u32x4 __attribute__((ext_vector_type(4)));

// 8 elements of a row from element k on (k + 8 <= K: K is a multiple of 32), any alignment.
template <int XT>
__device__ __forceinline__ void load8(const uint8_t* row, int64_t k, float (&x)[8]) {
  if constexpr (XT == F32) {
    z_u32x4 v[2];
    __builtin_memcpy(v, row + 4 * k, 32);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(v[e / 4][e % 4]);
  } else {
    z_u32x4 v;
    __builtin_memcpy(&v, row + 2 * k, 16);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = (v[e >> 1] >> (16 * (e & 1))) & 0xffffu;
      x[e] = XT == F16 ? f16_bits_to_float(h) : bf16_bits_to_float(h);
    }
  }
}

// UNROLL: groups of 512 elements a wave takes of a row together.
template <int XT, int UNROLL>
__global__ __launch_bounds__(256) void quantize_mx_kernel(QuantizeMxArgs p, int64_t first, int per) {
  constexpr int ES = DTypeInfo<XT>::bytes;
  const int lane = threadIdx.x & 63;
  const int64_t item = (first + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = item / per;
  if (t >= p.M) return;
  const int64_t k0 = (item - t * per) * (512 * UNROLL) + 8 * lane;
  const uint8_t* const src = reinterpret_cast<const uint8_t*>(p.X) + t * p.ldx * ES;
  float x[UNROLL][8];
  uint32_t code[UNROLL], byte[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    if (k0 + 512 * u < p.K) {
      load8<XT>(src, k0 + 512 * u, x[u]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[u][e] = 0.0f;
    }
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    // the bits of |x| are in the order of the values, infinity and NaN above them
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[u][e]) & 0x7fffffffu);
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xb1, 0xf, 0xf, false));  // lanes 1 0 3 2
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4e, 0xf, 0xf, false));  // lanes 2 3 0 1
    const uint32_t field = m >> 23;  // floor(log2 max) + 127
    const bool bad = field == 255u;
    byte[u] = bad ? 255u : field > 2u ? field - 2u : 0u;
    // A block of very small numbers: both sides 2^96 times larger, exactly, so that neither the numbers
    // nor the power of two are subnormal.
    const bool tiny = byte[u] < 27u;
    const float up = tiny ? 0x1p96f : 1.0f;
    const float scale = __uint_as_float((bad ? 127u : byte[u] + (tiny ? 96u : 0u)) << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[u][0] * up, x[u][1] * up, scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[u][2] * up, x[u][3] * up, scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[u][4] * up, x[u][5] * up, scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[u][6] * up, x[u][7] * up, scale, 3);
    code[u] = bad ? 0u : c;
  }
  for (int j = 0; j < p.top; ++j) {
    const int64_t at = p.place ? p.place[t * p.top + j] : t;
    if (at < 0 || at >= p.R) continue;
    uint8_t* const q = p.Q + at * p.ldq;
    uint8_t* const s = p.S + at * p.lds;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int64_t k = k0 + 512 * u;
      if (k >= p.K) continue;
      __builtin_memcpy(q + k / 2, &code[u], 4);
      if ((lane & 3) == 0) s[k / 32] = (uint8_t)byte[u];
    }
  }
}

template <int XT, int UNROLL>
hipError_t launch_unroll(const QuantizeMxArgs& p, hipStream_t s) {
  const int64_t per = ((int64_t)p.K + 512 * UNROLL - 1) / (512 * UNROLL);
  return launch_in_slices((p.M * per + 3) / 4, 256, [&](int64_t first, unsigned n) {
    hipLaunchKernelGGL((quantize_mx_kernel<XT, UNROLL>), dim3(n), dim3(256), 0, s, p, first, (int)per);
  });
}

// Two groups of 512 elements a wave, one where the row has no second (bf16, 16384 x 4096: 33.8 us with one,
// 29.5 with two, 33.3 with four; 65536 x 512: 15.7, 17.1, 24.6; 1 x 8192: 2.6, 2.5, 2.7).
template <int XT>
hipError_t launch_type(const QuantizeMxArgs& p, hipStream_t s) {
  return p.K <= 512 ? launch_unroll<XT, 1>(p, s) : launch_unroll<XT, 2>(p, s);
}

}  // namespace

hipError_t launch_quantize_mx(const QuantizeMxArgs& p, int x_type, hipStream_t s) {
  switch (x_type) {
    case F32: return launch_type<F32>(p, s);
    case F16: return launch_type<F16>(p, s);
    case BF16: return launch_type<BF16>(p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tgemm
