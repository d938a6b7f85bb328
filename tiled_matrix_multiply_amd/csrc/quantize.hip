// Rows in 8-bit integers with a scale each: scale = max |x| / 127, code = x / scale rounded to
// the nearest integer, ties to even.
#include "common.hpp"

namespace tgemm {

namespace {

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

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  return (a != a) ? a : (b != b) ? b : (a > b ? a : b);
}

template <int XT>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const void* X, int64_t ldx, int M, int K,
                                                            int8_t* Q, int64_t ldq, float* scales) {
  __shared__ float part[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    float m = 0.0f;
    for (int64_t k = tid; k < K; k += 256) m = max_nan(m, fabsf(load_as_float<XT>(X, row * ldx + k)));
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) m = max_nan(m, __shfl_xor(m, d));
    __syncthreads();  // the previous row's maxima have been read
    if (lane == 0) part[wave] = m;
    __syncthreads();
    m = max_nan(max_nan(part[0], part[1]), max_nan(part[2], part[3]));
    const float s = m / 127.0f;
    if (tid == 0) scales[row] = s;
    const bool live = s > 0.0f && s < __builtin_inff();
    const float k2 = prescale(s), sk = s * k2, r = 1.0f / sk;
    for (int64_t k = tid; k < K; k += 256)
      Q[row * ldq + k] = live ? (int8_t)code_of(load_as_float<XT>(X, row * ldx + k) * k2, sk, r) : (int8_t)0;
  }
}

}  // namespace

hipError_t launch_quantize_rows(const void* X, int64_t ldx, int M, int K, int x_type, int8_t* Q, int64_t ldq,
                                float* scales, hipStream_t s) {
  const unsigned grid = (unsigned)(M < (1 << 20) ? M : (1 << 20));
  switch (x_type) {
    case F32: hipLaunchKernelGGL((quantize_rows_kernel<F32>), dim3(grid), dim3(256), 0, s, X, ldx, M, K, Q, ldq, scales); break;
    case F16: hipLaunchKernelGGL((quantize_rows_kernel<F16>), dim3(grid), dim3(256), 0, s, X, ldx, M, K, Q, ldq, scales); break;
    case BF16: hipLaunchKernelGGL((quantize_rows_kernel<BF16>), dim3(grid), dim3(256), 0, s, X, ldx, M, K, Q, ldq, scales); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace tgemm
