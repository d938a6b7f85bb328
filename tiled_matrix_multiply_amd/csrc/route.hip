// Routing to experts: scores, the choice of the experts of each token, and the order of the rows that
// go to them; and the gradient of the logits.
//
// A token belongs to L lanes of a wave, each of them holding V neighbouring experts (L V >= E), so that
// the order of lanes is the order of experts: of equal keys the lowest lane's first one is the lower
// expert.  `top` rounds of a maximum over the lanes choose the experts; what a lane has lost in a round
// it takes out of its own values.
//
// The order of the rows needs no sorting: within a workgroup of up to 64 tokens each expert has a mask
// with a bit for each token (set in any order, the same in the end), and a pair's rank there is the
// number of bits below its own.  Up to 64 tokens are one workgroup and one launch.  More leave a
// table of blocks x experts counts (a byte each, at most 64), from which a second kernel takes where
// each block's rows start.
#include "experts.hpp"

namespace tgemm {

namespace {

typedef uint32_t r_u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float load_logit(const void* x, int64_t i, int type) {
  if (type == F32) return reinterpret_cast<const float*>(x)[i];
  const uint32_t h = reinterpret_cast<const uint16_t*>(x)[i];
  return type == F16 ? f16_bits_to_float(h) : bf16_bits_to_float(h);
}

constexpr float kNone = -__builtin_inff();

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xf, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xf, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float lane_value(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
__device__ __forceinline__ double lane_value(double v, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, l), hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// f over the L lanes of a token (16 or 64), in every one of them, in a fixed order: rotations within
// 16 lanes, then the four sixteens.
template <int L, class S, class F>
__device__ __forceinline__ S across(S v, F f) {
  v = f(v, dpp<0x128>(v));  // row_ror 8, 4, 2, 1
  v = f(v, dpp<0x124>(v));
  v = f(v, dpp<0x122>(v));
  v = f(v, dpp<0x121>(v));
  if constexpr (L == 64) v = f(f(lane_value(v, 0), lane_value(v, 16)), f(lane_value(v, 32), lane_value(v, 48)));
  return v;
}
template <int L, class S>
__device__ __forceinline__ S max_across(S v) {
  return across<L>(v, [](S a, S b) { return a > b ? a : b; });
}
template <int L, class S>
__device__ __forceinline__ S sum_across(S v) {
  return across<L>(v, [](S a, S b) { return a + b; });
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// The L lanes' part of a wave's ballot.
template <int L>
__device__ __forceinline__ uint64_t own_bits(uint64_t ballot, int lane) {
  return L == 64 ? ballot : (ballot >> (lane & 48)) & 0xffffull;
}

// The two largest of a set, -infinity where it has fewer.
template <class S>
struct Best2 {
  S a, b;
  __device__ __forceinline__ void add(S v) {
    const S low = v < a ? v : a;
    a = v < a ? a : v;
    b = b < low ? low : b;
  }
};

// The choice of one token's experts: lane j of the token's L gets the j-th (-1: none) and its logit.
// x: the lane's logits, -infinity where there is no expert; keys are computed in type S.
template <int L, int V, class S>
__device__ __forceinline__ void choose(const RouteArgs& p, const float (&x)[V], int lane, int sub, S rcp_sum, float x_max,
                                       int& chosen, float& chosen_x) {
  constexpr S none = -(S)__builtin_inf();
  const int e0 = sub * V;
  auto score = [&](float v) {
    return p.score ? (S)1 / ((S)1 + exp_of(-(S)v)) : exp_of((S)v - (S)x_max) * rcp_sum;
  };
  S key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    S k = x[i];
    if (p.bias) {
      const float b = e0 + i < p.E ? p.bias[e0 + i] : kNone;
      k = x[i] == kNone || b == kNone ? none : score(x[i]) + (S)b;
    }
    key[i] = k != k ? -none : k;
  }
  if (p.groups > 1) {
    // What each run of experts is worth: in the lane h < groups of the token, and in turn of h + L, ...
    const int size = p.E / p.groups;
    const bool by_score = !p.bias && p.group_top == 2;
    S worth[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      worth[i] = by_score && key[i] != none ? score(x[i]) : key[i];
      if (worth[i] != worth[i]) worth[i] = -none;
    }
    constexpr int GL = 64 / L;  // up to 64 runs
    S total[GL];
#pragma unroll
    for (int q = 0; q < GL; ++q) total[q] = none;
    for (int g = 0; g < p.groups; ++g) {
      Best2<S> m{none, none};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = e0 + i;
        m.add(e >= g * size && e < (g + 1) * size ? worth[i] : none);
      }
      const S a = max_across<L>(m.a);
      // the lowest lane that holds it gives up its first
      const uint64_t own = own_bits<L>(__ballot(m.a == a), lane);
      const S second = max_across<L>(sub == (int)__builtin_ctzll(own | 1ull << 63) ? m.b : m.a);
      const S t = p.group_top == 2 && second != none ? a + second : a;
#pragma unroll
      for (int q = 0; q < GL; ++q)
        if (g == sub + q * L) total[q] = t;
    }
    uint64_t kept = 0;
    for (int r = 0; r < p.top_groups; ++r) {
      S m = total[0];
#pragma unroll
      for (int q = 1; q < GL; ++q) m = total[q] > m ? total[q] : m;
      m = max_across<L>(m);
      int g = 64;  // the lowest of the runs that are worth it
#pragma unroll
      for (int q = GL - 1; q >= 0; --q) {
        const uint64_t own = own_bits<L>(__ballot(total[q] == m), lane);
        if (own) g = q * L + __builtin_ctzll(own);
      }
      if (m == none) break;  // (all lanes of a token together)
      kept |= 1ull << g;
#pragma unroll
      for (int q = 0; q < GL; ++q)
        if (g == sub + q * L) total[q] = none;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!((kept >> min((e0 + i) / size, 63)) & 1)) key[i] = none;
  }
  chosen = -1;
  chosen_x = 0.0f;
  for (int j = 0; j < p.top; ++j) {
    S m = key[0];
    int at = 0;
    float xm = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (key[i] > m) {
        m = key[i];
        at = i;
        xm = x[i];
      }
    const S best = max_across<L>(m);
    const uint64_t own = own_bits<L>(__ballot(m == best), lane);
    const int first = __builtin_ctzll(own | 1ull << 63);
    const int from = (lane & ~(L - 1)) + first;
    const int e = __shfl(e0 + at, from);
    const float v = __shfl(xm, from);
    if (sub == j) {
      chosen = best == none ? -1 : e;
      chosen_x = v;
    }
    if (sub == first) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == at) key[i] = none;
    }
  }
}

// The scores' common parts over a token: the largest logit and, for softmax, the sum of exp(x - largest).
template <int L, int V, class S>
__device__ __forceinline__ S softmax_sum(const float (&x)[V], float& x_max) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, x[i]);
  x_max = max_across<L>(m);
  S sum = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) sum += x[i] == kNone ? (S)0 : exp_of((S)x[i] - (S)x_max);
  return sum_across<L>(sum);
}

// Weight of the lane's chosen expert among the token's: p.top lanes hold one each.
template <int L, int V>
__device__ __forceinline__ float weight_of(const RouteArgs& p, int chosen, float cx, float x_max, float sum) {
  const bool there = chosen >= 0;
  if (!p.renorm) {
    const float s = p.score ? 1.0f / (1.0f + expf(-cx)) : expf(cx - x_max) / sum;
    return there ? p.scale * s : 0.0f;
  }
  // Relative to the largest chosen logit, so that the sum is at least 1/2: exp(x - m) for softmax; for
  // sigmoid exp(x - m) / (1 + exp(x)) with m = min(largest, 0), the scores times exp(-m).
  const float top = max_across<L>(there ? (cx != cx ? __builtin_inff() : cx) : kNone);
  const float m = p.score ? fminf(top, 0.0f) : top;
  float s = 0.0f;
  if (there) s = !p.score ? expf(cx - m) : cx > 0.0f ? 1.0f / (1.0f + expf(-cx)) : expf(cx - m) / (1.0f + expf(cx));
  const float all = sum_across<L>(s);
  return there ? p.scale * (s / all) : 0.0f;
}

// THREADS: of a workgroup.  TB tokens of a workgroup, 64 / L of them to a wave at a time.
template <int L, int V, int THREADS>
__global__ __launch_bounds__(THREADS) void route_kernel(RouteArgs p, int TB) {
  __shared__ unsigned long long mask[1024];
  __shared__ int start[1024 + 1];
  __shared__ int16_t pick[64 * 32];
  __shared__ int part[THREADS / 64];
  const int tid = threadIdx.x, lane = tid & 63, sub = lane & (L - 1), wave = tid >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * TB;
  const int here = (int)min((int64_t)TB, p.T - t0);
  for (int e = tid; e < p.E; e += THREADS) mask[e] = 0ull;
  __syncthreads();
  constexpr int TW = 64 / L, STEP = THREADS / 64 * TW;
  for (int base = wave * TW; base < here; base += STEP) {  // (the same for all lanes of a wave)
    const int local = base + lane / L;
    const bool live = local < here;
    const int64_t t = t0 + (live ? local : here - 1);
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = sub * V + i;
      x[i] = e < p.E ? load_logit(p.x, t * p.ldx + e, p.x_type) : kNone;
    }
    float x_max = 0.0f;
    double sum = 1.0;
    if (!p.score && (!p.renorm || p.bias || (p.groups > 1 && p.group_top == 2))) sum = softmax_sum<L, V, double>(x, x_max);
    int chosen;
    float cx;
    choose<L, V, double>(p, x, lane, sub, 1.0 / sum, x_max, chosen, cx);
    const float w = weight_of<L, V>(p, chosen, cx, x_max, (float)sum);
    if (live && sub < p.top) {
      pick[local * p.top + sub] = (int16_t)chosen;
      const int64_t at = t * p.top + sub;
      p.expert[at] = chosen;
      p.weight[at] = w;
      if (chosen >= 0) atomicOr(&mask[chosen], 1ull << local);
    }
  }
  __syncthreads();
  if (!p.ws) {  // the only block: where each expert's rows start
    int carry = 0;
    for (int base = 0; base < p.E; base += THREADS) {
      const int e = base + tid;
      int v = e < p.E ? __popcll(mask[e]) : 0;
      const int own = v;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(v, d);
        if (lane >= d) v += u;
      }
      if (lane == 63) part[wave] = v;
      __syncthreads();
      int before = carry, all = 0;
      for (int w = 0; w < THREADS / 64; ++w) {
        if (w < wave) before += part[w];
        all += part[w];
      }
      if (e < p.E) {
        start[e] = before + v - own;
        p.offsets[e] = before + v - own;
      }
      carry += all;
      __syncthreads();
    }
    if (tid == 0) p.offsets[p.E] = carry;
  } else {
    uint8_t* const row = p.ws + blockIdx.x * route_row_bytes(p.E);
    for (int e = tid; e < route_row_bytes(p.E); e += THREADS) row[e] = e < p.E ? (uint8_t)__popcll(mask[e]) : 0;
  }
  for (int i = tid; i < here * p.top; i += THREADS) {
    const int e = pick[i], local = i / p.top;
    int at = -1;
    if (e >= 0) at = __popcll(mask[e] & ((1ull << local) - 1)) + (p.ws ? 0 : start[e]);
    p.place[t0 * p.top + i] = at;
  }
}

// The second kernel: places within a block become places in the whole.  Every workgroup adds up the
// table of counts, all blocks' and those before its own (the table is read from the L2).
__global__ __launch_bounds__(256) void route_place_kernel(RouteArgs p, int TB, int blocks) {
  __shared__ int total[1024], before[1024], start[1024];
  __shared__ int part[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b0 = (int)((int64_t)blockIdx.x * blocks / gridDim.x), b1 = (int)((int64_t)(blockIdx.x + 1) * blocks / gridDim.x);
  for (int e = tid; e < 1024; e += 256) total[e] = before[e] = 0;
  __syncthreads();
  const int64_t row = route_row_bytes(p.E);
  const int per = (int)(row / 16);  // 16 experts to a thread
  const int rows = 256 / per, c = tid % per, r = tid / per;
  if (r < rows) {
    int all[16] = {}, mine[16] = {};
    for (int b = r; b < blocks; b += rows) {
      r_u32x4 v;
      __builtin_memcpy(&v, p.ws + b * row + 16 * c, 16);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int n = (v[i / 4] >> (8 * (i % 4))) & 255;
        all[i] += n;
        mine[i] += b < b0 ? n : 0;
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      atomicAdd(&total[16 * c + i], all[i]);
      atomicAdd(&before[16 * c + i], mine[i]);
    }
  }
  __syncthreads();
  int carry = 0;
  for (int base = 0; base < p.E; base += 256) {
    const int e = base + tid;
    int v = e < p.E ? total[e] : 0;
    const int own = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(v, d);
      if (lane >= d) v += u;
    }
    if (lane == 63) part[wave] = v;
    __syncthreads();
    int b = carry, all = 0;
    for (int w = 0; w < 4; ++w) {
      if (w < wave) b += part[w];
      all += part[w];
    }
    if (e < p.E) {
      start[e] = b + v - own + before[e];
      if (blockIdx.x == 0) p.offsets[e] = b + v - own;
    }
    carry += all;
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) p.offsets[p.E] = carry;
  for (int b = b0; b < b1; ++b) {
    const int64_t t0 = (int64_t)b * TB;
    const int n = (int)min((int64_t)TB, p.T - t0) * p.top;
    for (int i = tid; i < n; i += 256) {
      const int64_t at = t0 * p.top + i;
      const int e = p.expert[at];
      if (e >= 0) p.place[at] += start[e];
    }
    __syncthreads();
    for (int e = tid; e < p.E; e += 256) start[e] += p.ws[b * row + e];
    __syncthreads();
  }
}

// The gradient.  With g_j = scale * dweight_j and w the weights without the scale:
//   renorm:      d/d log s_j = w_j * sum_i w_i (g_j - g_i)                 over the chosen
//   otherwise:   d/d log s_j = w_j g_j
// and through log s: sigmoid times 1 - s = sigmoid(-x); softmax unchanged with renorm (the sum of the
// scores cancels), without it
//   dx_e = s_e (g_e - sum_j g_j s_j) = s_e (g_e U + sum_j s_j (g_e - g_j)),   U = the sum of the others' s
// (g_e = 0 for what was not chosen).  Written as differences none of them cancels where one weight is
// near 1.
template <int L, int V>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs p) {
  constexpr int TW = 64 / L;
  __shared__ float row[4 * TW][L * V];
  const int tid = threadIdx.x, lane = tid & 63, sub = lane & (L - 1);
  const int64_t t = (int64_t)blockIdx.x * (4 * TW) + tid / L;
  const bool live = t < p.T;
  const int64_t tt = live ? t : p.T - 1;
  float* const mine = row[tid / L];
  // the chosen: lane j has the j-th
  int e = -1;
  float g = 0.0f, cx = kNone;
  if (sub < p.top) {
    e = p.expert[tt * p.top + sub];
    if (e < 0 || e >= p.E) e = -1;
    if (e >= 0) {
      g = p.scale * p.dw[tt * p.top + sub];
      cx = load_logit(p.x, tt * p.ldx + e, p.x_type);
    }
  }
  const bool full = !p.score && !p.renorm;  // every logit has a gradient
  float s_all[V], sum = 1.0f, x_max = 0.0f, others = 0.0f;
  if (full) {
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = sub * V + i;
      x[i] = k < p.E ? load_logit(p.x, tt * p.ldx + k, p.x_type) : kNone;
    }
    sum = softmax_sum<L, V, float>(x, x_max);
    uint32_t taken = 0;  // which of the lane's experts were chosen
    for (int j = 0; j < p.top; ++j) {
      const int k = __shfl(e, (lane & ~(L - 1)) + j);
      if (k >= 0 && k / V == sub) taken |= 1u << (k % V);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s_all[i] = x[i] == kNone ? 0.0f : expf(x[i] - x_max) / sum;
      if (!((taken >> i) & 1)) others += s_all[i];
    }
    others = sum_across<L>(others);
  }
  float s;  // of the chosen, relative to a common factor with renorm
  if (p.renorm) {
    const float top = max_across<L>(e >= 0 ? (cx != cx ? __builtin_inff() : cx) : kNone);
    const float m = p.score ? fminf(top, 0.0f) : top;
    s = !p.score ? expf(cx - m) : cx > 0.0f ? 1.0f / (1.0f + expf(-cx)) : expf(cx - m) / (1.0f + expf(cx));
    if (e < 0) s = 0.0f;
    s = s / sum_across<L>(s);
  } else {
    s = p.score ? 1.0f / (1.0f + expf(-cx)) : expf(cx - x_max) / sum;
  }
  if (e < 0) s = 0.0f;
  float d = 0.0f, dot = 0.0f;
  for (int j = 0; j < p.top; ++j) {
    const int from = (lane & ~(L - 1)) + j;
    const float sj = __shfl(s, from), gj = __shfl(g, from);
    const bool there = __shfl(e, from) >= 0;
    if (there) {
      d += sj * (g - gj);
      dot += sj * gj;
    }
  }
  if (full) d = s * fmaf(g, others, d);
  else if (p.renorm) d = s * d;
  else d = s * g;
  if (p.score) d *= 1.0f / (1.0f + expf(cx));
#pragma unroll
  for (int i = 0; i < V; ++i) mine[sub * V + i] = full ? -s_all[i] * dot : 0.0f;
  __syncthreads();
  if (e >= 0) mine[e] = cx == kNone ? 0.0f : d;
  __syncthreads();
  if (!live) return;
  for (int k = sub; k < p.E; k += L) {
    const int64_t at = t * p.ldd + k;
    if (p.x_type == F32) store_from_float<F32>(p.dx, at, mine[k]);
    else if (p.x_type == F16) store_from_float<F16>(p.dx, at, mine[k]);
    else store_from_float<BF16>(p.dx, at, mine[k]);
  }
}

template <int L, int V, int THREADS>
hipError_t route_launch(const RouteArgs& p, int TB, hipStream_t s) {
  const int64_t blocks = p.T ? ((int64_t)p.T + TB - 1) / TB : 1;  // without tokens the offsets are written
  hipLaunchKernelGGL((route_kernel<L, V, THREADS>), dim3((unsigned)blocks), dim3(THREADS), 0, s, p, TB);
  return hipGetLastError();
}

}  // namespace

// (Work items of a launch are counted in 32 bits: at most 2^29 tokens, 64 to a workgroup of 256 threads.)
hipError_t launch_route(const RouteArgs& p, hipStream_t s) {
  const int TB = route_block_tokens(p.T);
  hipError_t e;
  const bool one = p.T <= 64;
  // 16 lanes to a token hold a choice of at most 16
  if (p.E <= 16) e = one ? route_launch<16, 1, 1024>(p, TB, s) : route_launch<16, 1, 256>(p, TB, s);
  else if (p.E <= 64 && p.top <= 16) e = one ? route_launch<16, 4, 1024>(p, TB, s) : route_launch<16, 4, 256>(p, TB, s);
  else if (p.E <= 256) e = one ? route_launch<64, 4, 1024>(p, TB, s) : route_launch<64, 4, 256>(p, TB, s);
  else e = one ? route_launch<64, 16, 1024>(p, TB, s) : route_launch<64, 16, 256>(p, TB, s);
  if (e != hipSuccess || one) return e;
  const int64_t blocks = route_blocks(p.T);
  hipLaunchKernelGGL(route_place_kernel, dim3((unsigned)(blocks < 256 ? blocks : 256)), dim3(256), 0, s, p, TB, (int)blocks);
  return hipGetLastError();
}

template <int L, int V>
static hipError_t grad_launch(const RouteGradArgs& p, hipStream_t s) {
  constexpr int TB = 4 * (64 / L);
  return launch_in_slices(((int64_t)p.T + TB - 1) / TB, 256, [&](int64_t first, unsigned n) {
    RouteGradArgs q = p;
    const int64_t t0 = first * TB;
    q.x = reinterpret_cast<const uint8_t*>(p.x) + t0 * p.ldx * (p.x_type == F32 ? 4 : 2);
    q.dx = reinterpret_cast<uint8_t*>(p.dx) + t0 * p.ldd * (p.x_type == F32 ? 4 : 2);
    q.expert += t0 * p.top;
    q.dw += t0 * p.top;
    q.T = (int)(p.T - t0);
    hipLaunchKernelGGL((route_grad_kernel<L, V>), dim3(n), dim3(256), 0, s, q);
  });
}

hipError_t launch_route_grad(const RouteGradArgs& p, hipStream_t s) {
  if (p.E <= 32 && p.top <= 16) return grad_launch<16, 2>(p, s);
  if (p.E <= 256 && p.top <= 16) return grad_launch<16, 16>(p, s);
  if (p.E <= 256) return grad_launch<64, 4>(p, s);
  return grad_launch<64, 16>(p, s);
}

}  // namespace tgemm
