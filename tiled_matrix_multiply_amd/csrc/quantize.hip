// Rows in 8-bit integers with a scale each: scale = max |x| / 127, code = x / scale rounded to
// the nearest integer, ties to even.
//
// One pass: the threads of a row hold it in registers between the maximum and the codes, 16 bytes
// a load, so that X is read once and Q written once; that is what bounds it (8191 x 8192: 37 to 38 us
// from fp16, 5.3 TB/s, 66 from fp32, 5.1).  Only what a row has beyond the registers (the loop after
// the first NV chunks of each thread) is read again.
#include <type_traits>

#include "common.hpp"

namespace tgemm {

namespace {

typedef uint32_t q_u32x4 __attribute__((ext_vector_type(4)));

// The code of x, the exact quotient x / s rounded to nearest, ties to even.
// r approximates 1 / s, so q is the right integer or a neighbour; the remainder x - q s is exact
// in fp32 (a multiple of the smaller operand's last place, below s in size) and decides.
__device__ __forceinline__ int code_of(float x, float s, float r) {
  float q = rintf(x * r);
  const float e = fmaf(-q, s, x), t = 2.0f * e;
  const bool odd = ((int)q & 1) != 0;
  if (t > s || (t == s && odd)) q += 1.0f;
  else if (t < -s || (t == -s && odd)) q -= 1.0f;
  return (int)fminf(fmaxf(q, -127.0f), 127.0f);
}

// A scale below 2^-100 would leave its reciprocal or the remainder outside the normal range:
// both sides of the quotient are then taken 2^64 times larger, which is exact.
__device__ __forceinline__ float prescale(float s) { return s < 0x1p-100f ? 0x1p64f : 1.0f; }

template <int XT>
struct QCfg {
  static constexpr int ES = DTypeInfo<XT>::bytes, CE = 16 / ES;  // elements of a chunk
};

// |x| as its bits, whose order as integers is the order of the values, with infinity above them
// and NaN above infinity: an integer maximum keeps a NaN.
template <int XT>
__device__ __forceinline__ uint32_t max_bits(q_u32x4 v) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (XT == F32) m = max(m, v[e] & 0x7fffffffu);
    else m = max(max(m, v[e] & 0x7fffu), (v[e] >> 16) & 0x7fffu);
  }
  return m;
}

template <int XT>
__device__ __forceinline__ float element(q_u32x4 v, int e) {
  if constexpr (XT == F32) return __uint_as_float(v[e]);
  const uint32_t h = (v[e >> 1] >> (16 * (e & 1))) & 0xffffu;
  return XT == F16 ? f16_bits_to_float(h) : bf16_bits_to_float(h);
}

// TPR: threads of a row (64: a wave, four rows a workgroup; 256: the workgroup).  NV: chunks of a
// thread held in registers.
template <int XT, int TPR, int NV>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const void* X, int64_t ldx, int M, int K,
                                                            int8_t* Q, int64_t ldq, float* scales) {
  constexpr int ES = QCfg<XT>::ES, CE = QCfg<XT>::CE;
  __shared__ uint32_t part[4];
  const int tid = threadIdx.x, t = tid % TPR;
  const int64_t row = (int64_t)blockIdx.x * (256 / TPR) + tid / TPR;
  if (TPR == 64 && row >= M) return;
  const uint8_t* const x = reinterpret_cast<const uint8_t*>(X) + row * ldx * ES;
  int8_t* const q = Q + row * ldq;
  auto fetch = [&](int64_t c) {  // chunk c of the row, zeros past its end
    q_u32x4 v = q_u32x4{0u, 0u, 0u, 0u};
    const int64_t k = c * CE;
    if (k + CE <= K) {
      __builtin_memcpy(&v, x + k * ES, 16);
    } else if (k < K) {
#pragma unroll
      for (int e = 0; e < CE; ++e)
        if (k + e < K) {
          if constexpr (ES == 4) v[e] = reinterpret_cast<const uint32_t*>(x)[k + e];
          else v[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(x)[k + e] << (16 * (e & 1));
        }
    }
    return v;
  };
  q_u32x4 v[NV];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = fetch(t + i * TPR);
#pragma unroll
  for (int i = 0; i < NV; ++i) m = max(m, max_bits<XT>(v[i]));
  const int64_t chunks = ((int64_t)K + CE - 1) / CE;
  for (int64_t c = t + NV * TPR; c < chunks; c += TPR) m = max(m, max_bits<XT>(fetch(c)));
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if constexpr (TPR > 64) {
    if ((tid & 63) == 0) part[tid >> 6] = m;
    __syncthreads();
    m = max(max(part[0], part[1]), max(part[2], part[3]));
  }
  float top;
  if constexpr (XT == F32) top = __uint_as_float(m);
  else top = XT == F16 ? f16_bits_to_float(m) : bf16_bits_to_float(m);
  const float s = top / 127.0f;
  if (t == 0) scales[row] = s;
  const bool live = s > 0.0f && s < __builtin_inff();
  const float up = prescale(s), su = s * up, r = 1.0f / su;
  const float half = live && up == 1.0f ? 0.5f * s : 0.0f;  // 0: every chunk takes the careful way
  // The codes of a chunk, the quick way: adding 1.5 * 2^23 to x r rounds it to an integer, which is
  // then the low byte of the sum's bits.  It is the code wherever the remainder x - q s stays
  // below s / 2 in size, which one maximum over the chunk tells; a tie, or a product x r that was
  // rounded across a border (both rare), sends the chunk through code_of.  About 6 vector
  // instructions an element instead of 20, which had taken longer than the memory: 8191 x 8192
  // fp16 rows 54.7 us before.
  auto codes = [&](q_u32x4 w, uint32_t (&o)[CE / 4]) {
    constexpr float kRound = 12582912.0f;
    float far = 0.0f;
    uint32_t b[CE];
#pragma unroll
    for (int e = 0; e < CE; ++e) {
      const float v = element<XT>(w, e), y = fmaf(v, r, kRound);
      far = fmaxf(far, fabsf(fmaf(-(y - kRound), s, v)));
      b[e] = __float_as_uint(y);
    }
    if (!(far < half)) {
#pragma unroll
      for (int e = 0; e < CE; ++e) b[e] = live ? (uint32_t)code_of(element<XT>(w, e) * up, su, r) : 0u;
    }
#pragma unroll
    for (int e = 0; e < CE; e += 4)
      o[e / 4] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[e + 3], b[e + 2], 0x0c0c0400u),
                                       __builtin_amdgcn_perm(b[e + 1], b[e], 0x0c0c0400u), 0x05040100u);
  };
  auto store = [&](int64_t c, q_u32x4 w) {
    const int64_t k = c * CE;
    if (k >= K) return;
    uint32_t o[CE / 4];
    codes(w, o);
    if (k + CE <= K) __builtin_memcpy(q + k, o, CE);
    else
      for (int e = 0; e < CE; ++e)
        if (k + e < K) q[k + e] = (int8_t)(o[e / 4] >> (8 * (e % 4)));
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) store(t + i * TPR, v[i]);
  for (int64_t c = t + NV * TPR; c < chunks; c += TPR) store(c, fetch(c));
}

template <int XT, int TPR, int NV>
hipError_t launch_rows(const void* X, int64_t ldx, int M, int K, int8_t* Q, int64_t ldq, float* scales, hipStream_t s) {
  constexpr int RPW = 256 / TPR;  // rows of a workgroup
  return launch_in_slices(((int64_t)M + RPW - 1) / RPW, 256, [&](int64_t first, unsigned n) {
    const int64_t row = first * RPW;
    hipLaunchKernelGGL((quantize_rows_kernel<XT, TPR, NV>), dim3(n), dim3(256), 0, s,
                       reinterpret_cast<const uint8_t*>(X) + row * ldx * QCfg<XT>::ES, ldx, (int)(M - row), K,
                       Q + row * ldq, ldq, scales + row);
  });
}

template <int XT>
hipError_t launch_type(const void* X, int64_t ldx, int M, int K, int8_t* Q, int64_t ldq, float* scales,
                       hipStream_t s) {
  // A wave holds a row of up to 64 x 4 chunks and needs no barrier; beyond, four waves share one.
  const int64_t chunks = ((int64_t)K + QCfg<XT>::CE - 1) / QCfg<XT>::CE;
  if (chunks <= 64 * 4) return launch_rows<XT, 64, 4>(X, ldx, M, K, Q, ldq, scales, s);
  if (chunks <= 256 * 4) return launch_rows<XT, 256, 4>(X, ldx, M, K, Q, ldq, scales, s);
  return launch_rows<XT, 256, 8>(X, ldx, M, K, Q, ldq, scales, s);
}

}  // namespace

hipError_t launch_quantize_rows(const void* X, int64_t ldx, int M, int K, int x_type, int8_t* Q, int64_t ldq,
                                float* scales, hipStream_t s) {
  switch (x_type) {
    case F32: return launch_type<F32>(X, ldx, M, K, Q, ldq, scales, s);
    case F16: return launch_type<F16>(X, ldx, M, K, Q, ldq, scales, s);
    case BF16: return launch_type<BF16>(X, ldx, M, K, Q, ldq, scales, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tgemm
