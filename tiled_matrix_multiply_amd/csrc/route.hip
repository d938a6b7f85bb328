// Routing to experts: scores, the choice of the experts of each token, and the order of the rows that
// go to them; and the gradient of the logits.
//
// A token belongs to L lanes of a wave, each of them holding V neighbouring experts (L V >= E), so that
// the order of lanes is the order of experts: of equal keys the lowest lane's first one is the lower
// expert.  Each lane sorts its keys once (as integers in the keys' order, with the place in the lane in
// their last bits), and `top` rounds of a maximum over the lanes' heads choose the experts.
//
// Keys are computed in fp32 with a bound on their error.  Where two neighbours in the order, or the last
// chosen and the first that was not, are nearer than the bound allows and not made of the same numbers,
// those few are ranked by keys in 64 bits; what that cannot settle (runs of experts that are worth the
// same, many near ones) is chosen again in 64 bits by the whole wave.
//
// The order of the rows needs no sorting: within a workgroup of up to 64 tokens each expert has a mask
// with a bit for each token (set in any order, the same in the end), and a pair's rank there is the
// number of bits below its own.  Some tokens (route_alone) are one workgroup and one launch.  More leave a
// table of blocks x experts counts (a byte each, at most 64), from which a second kernel takes where
// each block's rows start.
//
// What bounds it are chains of dependent steps, not the bytes: the logits' way from memory, `top` maxima across
// lanes, the counts' way through memory to the second kernel.  One token of 256 experts (sigmoid, bias, 4 of 8
// groups) 7.0 us, 8191 tokens 17 (13.6 and 5.0 by themselves; 8.4 MB, 2 us at the rate of a copy), 16384 of 128
// (softmax) 14.3.
#include "experts.hpp"
#include "grouped.hpp"

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

__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// The two largest of a set without NaN, -infinity where it has fewer.
template <class S>
struct Best2 {
  S a, b;
  __device__ __forceinline__ void add(S v) {
    if constexpr (sizeof(S) == 4) {
      b = __builtin_amdgcn_fmed3f(a, b, v);
      a = v > a ? v : a;
    } else {
      const S low = v < a ? v : a;
      a = v < a ? a : v;
      b = b < low ? low : b;
    }
  }
};

// Integers in the order of the values; 0 is below all of them.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true));
}
template <int L>
__device__ __forceinline__ uint32_t max_across(uint32_t v) {
  v = max_dpp<0x128>(v);
  v = max_dpp<0x124>(v);
  v = max_dpp<0x122>(v);
  v = max_dpp<0x121>(v);
  if constexpr (L == 64)
    v = max(max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16)),
            max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48)));
  return v;
}

// Falling order, by Batcher's odd-even merging of runs (63 exchanges for 16 values, two instructions each).
template <int V>
__device__ __forceinline__ void sort_falling(uint32_t (&v)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t a = v[i + j], b = v[i + j + k];
            v[i + j] = max(a, b);
            v[i + j + k] = min(a, b);
          }
}

// The lowest lane of a token's L (as an index among them) where `mine` holds; some lane's has to.
template <int L>
__device__ __forceinline__ int first_lane(bool mine, int lane) {
  const uint64_t m = __ballot(mine);
  if constexpr (L == 64) return (int)__builtin_ctzll(m);
  const uint32_t half = lane & 32 ? (uint32_t)(m >> 32) : (uint32_t)m;
  return (int)__builtin_ctz(half >> (lane & 16));
}

__device__ __forceinline__ float quick_exp(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504f); }

// The sum of a lane's values, pairwise.
template <int V>
__device__ __forceinline__ float lane_sum(const float (&v)[V]) {
  float s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = v[i];
#pragma unroll
  for (int d = 1; d < V; d *= 2)
#pragma unroll
    for (int i = 0; i + d < V; i += 2 * d) s[i] += s[i + d];
  return s[0];
}

// How a token's experts lie in its L lanes: each run of experts begins with a lane of its own and has a
// power of two of lanes, V experts to a lane, so that runs of any size meet in a few steps.  Without runs
// (or where they do not fit so) one after another.
struct Layout {
  int runs, size, lanes_log2;  // experts and lanes of a run
  __device__ __forceinline__ Layout(const RouteArgs& p, int run_lanes) {
    const bool apart = p.groups > 1 && run_lanes >= 0;
    runs = apart ? p.groups : 1;
    size = apart ? p.run_size : p.E;
    lanes_log2 = apart ? run_lanes : 6;
  }
  template <int V>
  __device__ __forceinline__ int in_run(int sub) const {
    return (sub & ((1 << lanes_log2) - 1)) * V;
  }
  template <int V>
  __device__ __forceinline__ int expert(int sub) const {  // the lane's first
    return (sub >> lanes_log2) * size + in_run<V>(sub);
  }
  template <int V>
  __device__ __forceinline__ int of_place(int q) const {  // the expert in place q % V of lane q / V
    return expert<V>(q / V) + q % V;
  }
  template <int V>
  __device__ __forceinline__ int count(int sub) const {  // and how many it has
    return (sub >> lanes_log2) < runs ? min(max(size - in_run<V>(sub), 0), V) : 0;
  }
};

// The n <= V logits of a lane from expert e on, -infinity after them.
template <int V>
__device__ __forceinline__ void load_logits(const void* logits, int64_t ldx, int type, int64_t t, int e, int n,
                                            float (&x)[V]) {
  const int64_t at = t * ldx + e;
  if (n == V && V > 1) {  // all loads together, of any alignment
    if (type == F32) {
      __builtin_memcpy(x, reinterpret_cast<const float*>(logits) + at, 4 * V);
    } else {
      uint32_t w[(V + 1) / 2] = {};
      __builtin_memcpy(w, reinterpret_cast<const uint16_t*>(logits) + at, 2 * V);
      if (type == F16) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = f16_bits_to_float((w[i / 2] >> (16 * (i & 1))) & 0xffffu);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = bf16_bits_to_float((w[i / 2] >> (16 * (i & 1))) & 0xffffu);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = i < n ? load_logit(logits, at + i, type) : kNone;
  }
}

// n <= V results of a lane from element `at` on, rounded once; all together where there are V, of any
// alignment.
template <int CT, int V>
__device__ __forceinline__ void store_run(void* to, int64_t at, int n, const float (&v)[V]) {
  if (n == V && V > 1) {
    if constexpr (CT == F32) {
      __builtin_memcpy(reinterpret_cast<float*>(to) + at, v, 4 * V);
    } else {
      uint32_t w[(V + 1) / 2] = {};
#pragma unroll
      for (int i = 0; i < V; ++i) w[i / 2] |= (CT == F16 ? float_to_f16_bits(v[i]) : float_to_bf16_bits(v[i])) << (16 * (i & 1));
      __builtin_memcpy(reinterpret_cast<uint16_t*>(to) + at, w, 2 * V);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) store_from_float<CT>(to, at + i, v[i]);
  }
}

// Whether the lane's run of experts is kept.  w: the two best of the lane; a run's worth is off by at
// most half of `slack`; sure turns false where that could decide.  A run's rank is the number of runs that
// are worth more: the 16 lanes of a token are turned by its length, of 64 one lane of each run is read.
template <int L, bool EXACT, class S>
__device__ __forceinline__ bool keep_run(const RouteArgs& p, int lm, Best2<S> w, int sub, S slack, bool& sure) {
  constexpr S none = -(S)__builtin_inf();
  auto meet = [&](S a, S b) {
    w.add(a);
    w.add(b);
  };
  const int m = 1 << lm;
  if (lm > 0) meet(dpp<0xb1>(w.a), dpp<0xb1>(w.b));    // lanes 1 0 3 2
  if (lm > 1) meet(dpp<0x4e>(w.a), dpp<0x4e>(w.b));    // lanes 2 3 0 1
  if (lm > 2) meet(dpp<0x141>(w.a), dpp<0x141>(w.b));  // eight lanes mirrored: the other four
  if (lm > 3) meet(dpp<0x140>(w.a), dpp<0x140>(w.b));  // sixteen mirrored: the other eight
  if constexpr (L == 64) {
    if (lm > 4) meet(__shfl_xor(w.a, 16), __shfl_xor(w.b, 16));
    if (lm > 5) meet(__shfl_xor(w.a, 32), __shfl_xor(w.b, 32));
  }
  // Sums of two keys in fp32 are taken in halves: that of two of the type's lowest numbers is a number then, and
  // not the -infinity of a run without experts.
  S t = w.a;
  if (p.group_top == 2) {
    constexpr S part = EXACT ? (S)1 : (S)0.5;
    t = part * w.a + (w.b != none ? part * w.b : (S)0);
    slack *= part;
  }
  const int first = sub & ~(m - 1);
  int over = 0, near = 0;  // runs that are worth more for certain, and those that may be
  auto rank = [&](S u, int from) {
    if constexpr (EXACT) {
      over += u > t || (u == t && from < first);
    } else {
      over += u - t > slack;
      near += !(u - t < -slack);
    }
  };
  if constexpr (L == 64) {
    for (int g = 0; g < p.groups; ++g) rank(lane_value(t, g << lm), g << lm);
    near -= 1;  // (its own)
  } else {
#define TGEMM_TURN(r) rank(dpp<0x120 + r>(t), (sub - r) & 15)
    if (lm < 1) {
      TGEMM_TURN(1); TGEMM_TURN(3); TGEMM_TURN(5); TGEMM_TURN(7); TGEMM_TURN(9); TGEMM_TURN(11); TGEMM_TURN(13); TGEMM_TURN(15);
    }
    if (lm < 2) {
      TGEMM_TURN(2); TGEMM_TURN(6); TGEMM_TURN(10); TGEMM_TURN(14);
    }
    if (lm < 3) {
      TGEMM_TURN(4); TGEMM_TURN(12);
    }
    if (lm < 4) TGEMM_TURN(8);
#undef TGEMM_TURN
  }
  if (EXACT) near = over;
  if (t == none) return false;  // no expert there
  if (over < p.top_groups && near >= p.top_groups) sure = false;
  return near < p.top_groups;
}

// The choice of one token's experts with keys in 64 bits, by a whole wave: lane j gets the j-th (-1: none)
// and its logit.  x: the lane's logits, -infinity where there is no expert.
template <int V>
__device__ __forceinline__ void choose(const RouteArgs& p, const Layout& lay, const float (&x)[V], int lane,
                                       double rcp_sum, float x_max, int& chosen, float& chosen_x) {
  constexpr double none = -__builtin_inf();
  const int e0 = lay.expert<V>(lane), n = lay.count<V>(lane);
  const bool by_score = !p.bias && p.groups > 1 && p.group_top == 2;
  double key[V], s[V];
  if (p.bias || by_score) {
    if (p.score) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = 1.0 / (1.0 + exp(-(double)x[i]));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = exp((double)x[i] - (double)x_max) * rcp_sum;
    }
  }
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float b = i < n ? p.bias[e0 + i] : kNone;
      const double k = s[i] + (double)b;
      key[i] = x[i] == kNone || b == kNone ? none : k;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = x[i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = key[i] != key[i] ? -none : key[i];
  double worth[V];  // of the expert to its run
#pragma unroll
  for (int i = 0; i < V; ++i) worth[i] = key[i];
  if (by_score) {
#pragma unroll
    for (int i = 0; i < V; ++i) worth[i] = key[i] == none ? none : s[i] != s[i] ? -none : s[i];
  }
  if (lay.runs > 1) {
    Best2<double> w{none, none};
#pragma unroll
    for (int i = 0; i < V; ++i) w.add(worth[i]);
    bool sure;
    if (!keep_run<64, true, double>(p, lay.lanes_log2, w, lane, 0.0, sure)) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = none;
    }
  } else if (p.groups > 1) {
    // Runs that do not fit the lanes, one after another: lane h < groups gets what run h is worth.
    const int size = p.run_size;
    double total = none;
    for (int g = 0; g < p.groups; ++g) {
      Best2<double> m{none, none};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = e0 + i;
        m.add(e >= g * size && e < (g + 1) * size ? worth[i] : none);
      }
      const double a = max_across<64>(m.a);
      // the lowest lane that holds it gives up its first
      const double second = max_across<64>(lane == (int)__builtin_ctzll(__ballot(m.a == a)) ? m.b : m.a);
      if (g == lane) total = p.group_top == 2 && second != none ? a + second : a;
    }
    uint64_t kept = 0;
    for (int r = 0; r < p.top_groups; ++r) {
      const double m = max_across<64>(total);
      if (m == none) break;
      const int g = (int)__builtin_ctzll(__ballot(total == m));  // the lowest of the runs that are worth it
      kept |= 1ull << g;
      if (g == lane) total = none;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!((kept >> min((e0 + i) / size, 63)) & 1)) key[i] = none;
  }
  chosen = -1;
  chosen_x = 0.0f;
  for (int j = 0; j < p.top; ++j) {
    double m = key[0];
    int at = 0;
    float xm = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (key[i] > m) {
        m = key[i];
        at = i;
        xm = x[i];
      }
    const double best = max_across<64>(m);
    const int first = (int)__builtin_ctzll(__ballot(m == best));
    const int e = __builtin_amdgcn_readlane(e0 + at, first);
    const float v = lane_value(xm, first);
    if (lane == j) {
      chosen = best == none ? -1 : e;
      chosen_x = v;
    }
    if (lane == first) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == at) key[i] = none;
    }
  }
}

// ---- the same in fp32, where that is certain ----

// choose() in fp32: lane j of the token's L gets the place (lane * V + i) of the j-th, -1 for none, and its
// logit; false in the lanes of a token for which fp32 is not enough.
// logits: the token's in LDS, by place, and biases alike; record: L + 1 of the token's own in LDS.
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));
template <int L, int V>
__device__ __forceinline__ bool choose_quick(const RouteArgs& p, const Layout& lay, const float (&x)[V],
                                             const float (&bias)[V], const float* logits,
                                             const float* biases, u2_t* record, int lane, int sub,
                                             float x_max, float rcp_sum, int& chosen, float& chosen_x) {
  constexpr uint32_t LOW = V - 1;
  const bool scored = p.bias || (p.groups > 1 && p.group_top == 2);
  float key[V], s[V];
  float slack = 0.0f;  // bound on the error of a score
  if (scored) {
    // Relative errors: the exponential's argument is off by half a step or two of itself, the function
    // and the reciprocal by a step.  z exp(-z) <= 0.37, and z s(-z) falls from z = 1.3 on, so that the
    // argument's part is largest at the largest score.  softmax: its sum is off by up to 10 half steps.
    // Absolute: a sigmoid below 2^-126 is 0 here, and a softmax's bound is far above that.
    if (p.score) {
      slack = __builtin_amdgcn_rcpf(1.0f + quick_exp(-x_max)) * (0x1p-21f + fmaxf(1.3f, -x_max) * 0x1p-22f) + 0x1p-125f;
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = __builtin_amdgcn_rcpf(1.0f + quick_exp(-x[i]));
    } else {
      slack = rcp_sum * 0x1p-19f;
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = quick_exp(x[i] - x_max) * rcp_sum;
    }
  }
  constexpr float inf = __builtin_inff();
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float k = fminf(s[i] + bias[i], inf);  // a NaN as infinity
      key[i] = x[i] == kNone || bias[i] == kNone ? kNone : k;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = fminf(x[i] + 0.0f, inf);  // (one zero)
  }
  bool sure = true;
  uint32_t keep = ~LOW;
  if (p.groups > 1) {
    Best2<float> w{kNone, kNone};
    if (!p.bias && p.group_top == 2) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float v = fminf(s[i], inf);
        w.add(key[i] == kNone ? kNone : v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) w.add(key[i]);
    }
    // a run's sum of two: twice the error, and the roundings of the sum and of its keys
    const float worst = max_across<L>(fmaxf(w.a == kNone ? 0.0f : fabsf(w.a), w.b == kNone ? 0.0f : fabsf(w.b)));
    const bool kept = scored ? keep_run<L, false, float>(p, lay.lanes_log2, w, sub, 4.0f * slack + 0x1p-21f * worst, sure)
                             : keep_run<L, true, float>(p, lay.lanes_log2, w, sub, 0.0f, sure);
    if (!kept) keep = 0u;
  }
  // (-infinity, and whatever is not kept, is below FINITE)
  constexpr uint32_t FINITE = 0x00800000u;
  uint32_t u[V];
#pragma unroll
  for (int i = 0; i < V; ++i) u[i] = (ordered(key[i]) & keep) | (LOW - i);
  sort_falling<V>(u);
  // The best head of the token's lanes, the lowest lane's of equal ones (their last bits are places, not
  // values), becomes the token's j-th record and leaves its lane.
  auto next = [&](int j) {
    const uint32_t head = u[0] & ~LOW, best = max_across<L>(head);
    const bool own = sub == first_lane<L>(head == best, lane);
    if (own) record[j] = u2_t{best, (uint32_t)(sub * V) + LOW - (u[0] & LOW)};
    // (a mask that the compiler cannot see through: it would make a branch of the selects, with twice the moves)
    uint32_t all = own ? ~0u : 0u;
    asm volatile("" : "+v"(all));
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = (all & (i + 1 < V ? u[i + 1 < V ? i + 1 : i] : 0u)) | (~all & u[i]);
    return best;
  };
  auto apart = [&](uint32_t a, uint32_t b) {  // a >= b, without their last bits
    if (!p.bias) return a != b;  // the logits themselves
    // what the last bits were worth, and two roundings
    const float fa = from_ordered(a), fb = from_ordered(b);
    return fa - fb > 2.0f * slack + (V + 4) * 0x1p-23f * fmaxf(fabsf(fa), fabsf(fb));
  };
  uint32_t last = 0;
  for (int j = 0; j < p.top; ++j) last = next(j);
  // Those that were not chosen but may be worth as much as the last one come behind it, up to four and up to
  // the token's lanes: ranked below, no more than that, or one of them would get the place of another token's
  // first (where there are more, the token is chosen again).
  int found = p.top;
  if (last >= FINITE) {
    const int most = p.top + 4 < L ? p.top + 4 : L;
    for (;;) {
      const uint32_t r = next(found);
      if (r < FINITE || apart(last, r)) break;
      if (found == most) {
        sure = false;
        break;
      }
      ++found;
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const u2_t got = record[sub < found ? sub : 0];
  const bool there = sub < found && got[0] >= FINITE;
  const uint32_t mine = there ? got[0] : 0u;
  int place = there ? (int)got[1] : -1;
  // Is the order certain?  Neighbours have to be apart or made of the same numbers.
  float cx = place >= 0 ? logits[place] : 0.0f;
  const float cb = p.bias && place >= 0 ? biases[place] : 0.0f;
  const uint32_t u2 = (uint32_t)__shfl((int)mine, lane + 1);
  const bool same = __shfl(cx, lane + 1) == cx && __shfl(cb, lane + 1) == cb;
  const bool doubt = sub + 1 < found && u2 && !apart(mine, u2) && !same;
  const uint64_t all = __ballot(doubt);
  if (L == 64 ? all != 0 : ((all >> (lane & 48)) & 0xffff) != 0) {
    if (p.bias && !p.score) {
      sure = false;  // the softmax's sum would be needed in 64 bits
    } else {
      // the candidates' keys in 64 bits, and each one's rank among them
      double k = p.bias ? 1.0 / (1.0 + exp(-(double)cx)) + (double)cb : (double)cx;
      k = place < 0 ? -__builtin_inf() : k != k ? __builtin_inf() : k;
      int rank = 0;
      for (int j = 0; j < found; ++j) {
        const int from = (lane & ~(L - 1)) + j;
        const double kj = __shfl(k, from);
        const int pj = __shfl(place, from);
        rank += kj > k || (kj == k && (j < sub ? pj <= place : pj < place));
      }
      const int to = 4 * ((lane & ~(L - 1)) + (sub < found ? rank : sub));
      place = __builtin_amdgcn_ds_permute(to, place);
      cx = __int_as_float(__builtin_amdgcn_ds_permute(to, __float_as_int(cx)));
    }
  }
  chosen = sub < p.top ? place : -1;
  chosen_x = cx;
  return sure;
}

// The scores' common parts over a token: the largest logit and, for softmax, the sum of exp(x - largest).
// NaN is left out of the maximum on either side of each step, so that all lanes of the token get the same (a
// comparison would leave it out on one side only, and the bound on the keys' errors and the number of
// candidates, which go by this, would differ from lane to lane).
template <int L, int V>
__device__ __forceinline__ float largest(const float (&x)[V]) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, x[i]);
  return across<L>(m, [](float a, float b) { return fmaxf(a, b); });
}
template <int L, int V, class S>
__device__ __forceinline__ S softmax_sum(const float (&x)[V], float x_max) {
  if constexpr (sizeof(S) == 8) {
    S sum = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += x[i] == kNone ? (S)0 : exp_of((S)x[i] - (S)x_max);
    return sum_across<L>(sum);
  } else {
    float e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = x[i] == kNone ? 0.0f : expf(x[i] - x_max);
    return sum_across<L>(lane_sum<V>(e));
  }
}

// exp(v) within two steps, 0 below 2^-126: the product with log2(e) in two parts.
__device__ __forceinline__ float exp_near(float v) {
  constexpr float hi = 1.44269502f, lo = 1.92596299e-8f;  // log2(e) in two fp32 numbers
  const float t = v * hi, rest = fmaf(v, lo, fmaf(v, hi, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return fabsf(v) < 87.33f ? fmaf(e, rest * 0.693147181f, e) : e;  // (past 126 ln 2 e or the rest may be no number)
}

// A chosen score relative to the largest chosen logit, so that their sum is at least 1/2: exp(x - top) for
// softmax; for sigmoid exp(x - m) / (1 + exp(x)) with m = min(top, 0), the score times exp(-m).
__device__ __forceinline__ float score_near(int sigmoid, float x, float top) {
  if (!sigmoid) return exp_near(x - top);
  // x > 0: then m = 0 and the score is 1 / (1 + exp(-x))
  const float e = exp_near(x > 0.0f ? -x : x);
  return (x > 0.0f ? 1.0f : exp_near(x - fminf(top, 0.0f))) * __builtin_amdgcn_rcpf(1.0f + e);
}

// Weight of the lane's chosen expert among the token's: p.top lanes hold one each.  sum: of the softmax, or any
// number where nothing but the logits decided the choice (then NaN or +infinity is among the chosen).
template <int L, int V>
__device__ __forceinline__ float weight_of(const RouteArgs& p, int chosen, float cx, float x_max, float sum) {
  const bool there = chosen >= 0;
  if (!p.renorm) {
    const float s = p.score ? __builtin_amdgcn_rcpf(1.0f + exp_near(-cx)) : exp_near(cx - x_max) / sum;
    return there ? p.scale * s : 0.0f;
  }
  const float top = max_across<L>(there ? (cx != cx ? __builtin_inff() : cx) : kNone);
  float s = score_near(p.score, cx, top);
  if (!there) s = 0.0f;
  float all = sum_across<L>(s);
  // (a softmax over NaN or +infinity has no scores, also where the chosen logits, which are all that is read
  // here, are numbers)
  if (!p.score && sum != sum) all = sum;
  return there ? p.scale * (s / all) : 0.0f;
}

// One token again in 64 bits, by the whole wave: lane j < top gets the j-th expert and its logit.
// run_lanes: the layout's, for VV experts a lane.
template <int VV>
__device__ __forceinline__ void choose_again(const RouteArgs& p, int run_lanes, int64_t t, int lane, int& chosen,
                                             float& cx) {
  const Layout lay(p, run_lanes);
  float x[VV];
  load_logits<VV>(p.x, p.ldx, p.x_type, t, lay.expert<VV>(lane), lay.count<VV>(lane), x);
  float x_max = 0.0f;
  double sum = 1.0;
  if (!p.score && (p.bias || (p.groups > 1 && p.group_top == 2))) {
    x_max = largest<64, VV>(x);
    sum = softmax_sum<64, VV, double>(x, x_max);
  }
  choose<VV>(p, lay, x, lane, 1.0 / sum, x_max, chosen, cx);
}

// TB tokens of a workgroup, 64 / L of them to a wave at a time.
template <int L, int V, int THREADS>
__global__ __launch_bounds__(THREADS) void route_kernel(RouteArgs p, int TB) {
  __shared__ unsigned long long mask[1024];
  __shared__ int start[1024 + 1];
  __shared__ int16_t pick[64 * 32];
  __shared__ int part[THREADS / 64];
  __shared__ __attribute__((aligned(16))) float logits[THREADS / L][L * V];
  __shared__ __attribute__((aligned(16))) float biases[L * V];
  __shared__ u2_t record[THREADS / L][L + 1];
  constexpr int VV = (L * V + 63) / 64;
  const int tid = threadIdx.x, lane = tid & 63, sub = lane & (L - 1), wave = tid >> 6, threads = blockDim.x;
  const int64_t t0 = (int64_t)blockIdx.x * TB;
  const int here = (int)min((int64_t)TB, p.T - t0);
  constexpr int TW = 64 / L;
  const Layout lay(p, p.run_lanes);
  const int e0 = lay.expert<V>(sub), n = lay.count<V>(sub);
  float bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) bias[i] = kNone;
  if (p.bias) {
    if (n == V) {
      __builtin_memcpy(bias, p.bias + e0, 4 * V);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) bias[i] = p.bias[e0 + i];
    }
  }
  if (tid < L) {
#pragma unroll
    for (int i = 0; i < V; ++i) biases[sub * V + i] = bias[i];
  }
  for (int e = tid; e < p.E; e += threads) mask[e] = 0ull;
  __syncthreads();
  for (int base = wave * TW; base < here; base += threads / 64 * TW) {  // (the same for all lanes of a wave)
    const int local = base + lane / L;
    const bool live = local < here;
    const int64_t t = t0 + (live ? local : here - 1);
    float x[V];
    load_logits<V>(p.x, p.ldx, p.x_type, t, e0, n, x);
    const bool scored = p.bias || (p.groups > 1 && p.group_top == 2);
    float x_max = 0.0f, sum = 1.0f;
    if (scored || (!p.score && !p.renorm)) {
      x_max = largest<L, V>(x);
      if (!p.score) sum = softmax_sum<L, V, float>(x, x_max);
    }
    int chosen = -1;
    float cx = 0.0f;
    bool sure = false;
    if (p.run_lanes >= 0) {
      // the wave's own rows: its writes and reads of them keep their order
      float* const row = logits[tid / L];
#pragma unroll
      for (int i = 0; i < V; ++i) row[sub * V + i] = x[i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      int place;
      sure = choose_quick<L, V>(p, lay, x, bias, row, biases, record[tid / L], lane, sub, x_max, 1.0f / sum, place, cx);
      chosen = place >= 0 ? lay.of_place<V>(place) : -1;
    }
    for (uint64_t again = __ballot(!sure); again;) {
      const int from = (int)__builtin_ctzll(again) & ~(L - 1);  // the token's first lane
      again &= ~((L == 64 ? ~0ull : 0xffffull) << from);
      const int at = base + from / L;
      int c;
      float v;
      // (a quarter of the experts to a lane, so four times the lanes to a run)
      choose_again<VV>(p, p.run_lanes < 0 || L == 64 || V == 1 ? p.run_lanes : p.run_lanes + 2,
                       t0 + (at < here ? at : here - 1), lane, c, v);
      const int cs = __shfl(c, sub);
      const float vs = __shfl(v, sub);
      if ((lane & ~(L - 1)) == from) {
        chosen = cs;
        cx = vs;
      }
    }
    const float w = weight_of<L, V>(p, chosen, cx, x_max, sum);
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
    for (int base = 0; base < p.E; base += threads) {
      const int e = base + tid;
      int v = e < p.E ? __popcll(mask[e]) : 0;
      const int own = v;
      v = scan_add(v);
      if (lane == 63) part[wave] = v;
      __syncthreads();
      int before = carry, all = 0;
      for (int w = 0; w < threads / 64; ++w) {
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
    for (int e = tid; e < route_row_bytes(p.E); e += threads) row[e] = e < p.E ? (uint8_t)__popcll(mask[e]) : 0;
  }
  for (int i = tid; i < here * p.top; i += threads) {
    const int e = pick[i], local = (int)((uint32_t)(i * p.per_top) >> 16);
    int at = -1;
    if (e >= 0) at = __popcll(mask[e] & ((1ull << local) - 1)) + (p.ws ? 0 : start[e]);
    p.place[t0 * p.top + i] = at;
  }
}

// The second kernel: places within a block become places in the whole.  Every workgroup adds up the
// table of counts, all blocks' and those before its own (the table is read from the L2), 4 experts to a
// thread: bytes apart in sums of 16 bits, flushed before they could pass 65535 (1000 rows of at most 64).
// It is a chain of waits: the loads of a thread go out together, one pass gives both sums, nothing is divided
// but by powers of two (cols: threads to a row of the table), and long tables have 1024 threads (63 rows of 64
// bytes 3.4 us, 256 of 256 5.1; with divisions, two passes and 256 threads 5.4 and 7.1).
__global__ __launch_bounds__(1024) void route_place_kernel(RouteArgs p, int TB, int blocks, int cols) {
  __shared__ int total[1024], before[1024], start[1024];
  __shared__ int part[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, threads = blockDim.x;
  int b0 = blockIdx.x, b1 = b0 + 1;
  if ((int)gridDim.x < blocks) {  // (256 of them at most, and less than 2^23 blocks)
    b0 = (int)(blockIdx.x * (uint32_t)blocks / gridDim.x);
    b1 = (int)((blockIdx.x + 1) * (uint32_t)blocks / gridDim.x);
  }
  // the first block's pairs, fetched while the table is
  constexpr int AHEAD = 2;
  const int64_t at0 = (int64_t)b0 * TB * p.top;
  const int pairs0 = (int)min((int64_t)TB, p.T - (int64_t)b0 * TB) * p.top;
  int e_first[AHEAD], rank_first[AHEAD];
#pragma unroll
  for (int q = 0; q < AHEAD; ++q) {
    const int i = min(tid + threads * q, pairs0 - 1);
    e_first[q] = p.expert[at0 + i];
    rank_first[q] = p.place[at0 + i];
  }
  const int row = (int)route_row_bytes(p.E), lc = __builtin_ctz(cols), rows = threads >> lc;
  const int c = min(tid & (cols - 1), row / 4 - 1), r = tid >> lc;
  for (int e = tid; e < row; e += threads) total[e] = before[e] = 0;
  __syncthreads();
  for (int chunk = 0; chunk < blocks; chunk += 1000 * rows) {
    const int here = min(1000 * rows, blocks - chunk);  // rows of the table
    const uint8_t* const table = p.ws + (int64_t)chunk * row;
    uint32_t even = 0, odd = 0, even_b = 0, odd_b = 0;
    auto batch = [&](int b, auto count) {  // rows b + q * rows of the chunk
      constexpr int N = decltype(count)::value;
      uint32_t v[N];
#pragma unroll
      for (int q = 0; q < N; ++q)
        v[q] = *reinterpret_cast<const uint32_t*>(table + (uint32_t)(min(b + q * rows, here - 1) * row + 4 * c));
#pragma unroll
      for (int q = 0; q < N; ++q) {
        const int at = b + q * rows;
        const uint32_t w = at < here ? v[q] : 0u, e = w & 0x00ff00ffu, o = (w >> 8) & 0x00ff00ffu;
        even += e;
        odd += o;
        even_b += chunk + at < b0 ? e : 0u;
        odd_b += chunk + at < b0 ? o : 0u;
      }
    };
    if (here <= 4 * rows) {
      batch(r, std::integral_constant<int, 4>{});
    } else {
      for (int b = r; b - r < here; b += 16 * rows) batch(b, std::integral_constant<int, 16>{});
    }
    if ((tid & (cols - 1)) < row / 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        atomicAdd(&total[4 * c + i], (int)(((i & 1 ? odd : even) >> (8 * (i & 2))) & 0xffffu));
        if (b0 > 0) atomicAdd(&before[4 * c + i], (int)(((i & 1 ? odd_b : even_b) >> (8 * (i & 2))) & 0xffffu));
      }
    }
  }
  __syncthreads();
  int carry = 0;
  for (int base = 0; base < p.E; base += threads) {
    const int e = base + tid;
    const int own = e < p.E ? total[e] : 0, v = scan_add(own);
    if (lane == 63) part[wave] = v;
    __syncthreads();
    int b = carry, all = 0;
    for (int w = 0; w < threads / 64; ++w) {
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
    int done = 0;
    if (b == b0) {
#pragma unroll
      for (int q = 0; q < AHEAD; ++q)
        if (tid + threads * q < n && e_first[q] >= 0) p.place[at0 + tid + threads * q] = rank_first[q] + start[e_first[q]];
      done = threads * AHEAD;
    }
    for (int i = done + tid; i < n; i += threads) {
      const int64_t at = t0 * p.top + i;
      const int e = p.expert[at];
      if (e >= 0) p.place[at] += start[e];
    }
    if (b + 1 == b1) break;
    __syncthreads();
    for (int e = tid; e < p.E; e += threads) start[e] += p.ws[(int64_t)b * row + e];
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
// Its bytes bound it where there are many tokens: softmax as it is in fp32, 16384 x 128 6.4 us, 16384 x 512 13.9
// (4.8 TB/s).
// A token's row of results lies in LDS between what every expert gets and what the chosen get; only the
// wave that owns it touches it, so its writes and reads keep their order without a barrier.
__device__ __forceinline__ void row_written() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int L, int V>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs p) {
  constexpr int TW = 64 / L;
  __shared__ __attribute__((aligned(16))) float row[4 * TW][L * V];
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
    g = p.scale * p.dw[tt * p.top + sub];
    if (e >= 0 && e < p.E) cx = load_logit(p.x, tt * p.ldx + e, p.x_type);
    if (cx == kNone) {  // no expert, or none that could be chosen
      e = -1;
      g = 0.0f;
    }
  }
  const int e0 = sub * V, n = min(max(p.E - e0, 0), V);
  const bool full = !p.score && !p.renorm;  // every logit has a gradient
  float v[V], sum = 1.0f, x_max = 0.0f, others = 0.0f;
  if (full) {
    load_logits<V>(p.x, p.ldx, p.x_type, tt, e0, n, v);
    x_max = largest<L, V>(v);
    // the scores; then once more without the chosen's
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = v[i] == kNone ? 0.0f : exp_near(v[i] - x_max);
    sum = sum_across<L>(lane_sum<V>(v));
    const float r = sum == 0.0f ? 0.0f : 1.0f / sum;  // (a token that is masked as a whole)
#pragma unroll
    for (int i = 0; i < V; ++i) mine[e0 + i] = v[i] * r;
    row_written();
    if (e >= 0) mine[e] = 0.0f;
    row_written();
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = mine[e0 + i];
    others = sum_across<L>(lane_sum<V>(v));
  }
  float s;  // of the chosen, relative to a common factor with renorm
  if (p.renorm) {
    const float top = max_across<L>(e >= 0 ? (cx != cx ? __builtin_inff() : cx) : kNone);
    s = score_near(p.score, cx, top);
    if (e < 0) s = 0.0f;
    s = s / sum_across<L>(s);
  } else {
    s = p.score ? __builtin_amdgcn_rcpf(1.0f + exp_near(-cx)) : exp_near(cx - x_max) / sum;
  }
  if (e < 0) s = 0.0f;
  // sums over the chosen: of s (g_e - g) and of s g
  float d = 0.0f, dot = 0.0f;
  if constexpr (L == 64) {
    for (int j = 0; j < p.top; ++j) {
      const float sj = lane_value(s, j);
      d = fmaf(sj, g - lane_value(g, j), d);
    }
  } else {
#define TGEMM_TURN(r) d = fmaf(dpp<0x120 + r>(s), g - dpp<0x120 + r>(g), d)
    TGEMM_TURN(1); TGEMM_TURN(2); TGEMM_TURN(3); TGEMM_TURN(4); TGEMM_TURN(5);
    TGEMM_TURN(6); TGEMM_TURN(7); TGEMM_TURN(8); TGEMM_TURN(9); TGEMM_TURN(10);
    TGEMM_TURN(11); TGEMM_TURN(12); TGEMM_TURN(13); TGEMM_TURN(14); TGEMM_TURN(15);
#undef TGEMM_TURN
  }
  if (full) {
    dot = sum_across<L>(s * g);
    d = s * fmaf(g, others, d);
  } else {
    d = p.renorm ? s * d : s * g;
  }
  if (p.score) d *= __builtin_amdgcn_rcpf(1.0f + exp_near(cx));
#pragma unroll
  for (int i = 0; i < V; ++i) mine[e0 + i] = full ? -v[i] * dot : 0.0f;
  row_written();
  if (e >= 0) mine[e] = d;
  row_written();
  if (!live) return;
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = mine[e0 + i];
  const int64_t at = t * p.ldd + e0;
  if (p.x_type == F32) store_run<F32, V>(p.dx, at, n, v);
  else if (p.x_type == F16) store_run<F16, V>(p.dx, at, n, v);
  else store_run<BF16, V>(p.dx, at, n, v);
}

template <int L, int V, int MOST>
hipError_t route_launch(const RouteArgs& p, int TB, hipStream_t s) {
  const int64_t blocks = p.T ? ((int64_t)p.T + TB - 1) / TB : 1;  // without tokens the offsets are written
  // a workgroup's tokens all at once, if its waves can be that many
  const int tokens = p.T < TB ? p.T : TB;
  int threads = (tokens * L + 255) / 256 * 256;
  threads = threads < 256 ? 256 : threads > MOST ? MOST : threads;
  if (blocks * threads > 0xffffffffLL) threads = 256;  // the runtime counts work items in 32 bits
  hipLaunchKernelGGL((route_kernel<L, V, MOST>), dim3((unsigned)blocks), dim3(threads), 0, s, p, TB);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& args, hipStream_t s) {
  RouteArgs p = args;
  p.run_size = p.E / p.groups;
  p.per_top = (65536 + p.top - 1) / p.top;
  const int TB = route_block_tokens(p.T, p.E);
  // Lanes of a token: 16 hold a choice of at most 16 from at most 256 experts; up to 8 tokens of more than 128
  // are over sooner with 64 (4 x 256: 6.5 us against 7.0, 16 x 256 8.8 against 7.3; 4 x 128 6.8 against 6.1).
  // Experts of a lane: the fewest that hold all of them, runs of them in lanes of their own (2000 x 512
  // with 16 to a lane 24.0 us, with 8 17.7).
  auto fits = [&](int L, int V) {
    if (p.groups == 1) {
      p.run_lanes = 6;
      return p.E <= L * V;
    }
    const int size = p.run_size;
    p.run_lanes = 0;
    while ((V << p.run_lanes) < size) ++p.run_lanes;
    return p.groups << p.run_lanes <= L;
  };
  hipError_t e;
  if (p.top > 16 || !fits(16, 16) || (p.T <= 8 && !fits(16, 8)))
    e = fits(64, 1)    ? route_launch<64, 1, 1024>(p, TB, s)
        : fits(64, 4)  ? route_launch<64, 4, 1024>(p, TB, s)
        : fits(64, 8)  ? route_launch<64, 8, 1024>(p, TB, s)
        : fits(64, 16) ? route_launch<64, 16, 512>(p, TB, s)
                       : (p.run_lanes = -1, route_launch<64, 16, 512>(p, TB, s));  // all in 64 bits
  else
    e = fits(16, 1)   ? route_launch<16, 1, 1024>(p, TB, s)
        : fits(16, 4) ? route_launch<16, 4, 1024>(p, TB, s)
        : fits(16, 8) ? route_launch<16, 8, 1024>(p, TB, s)
                      : (fits(16, 16), route_launch<16, 16, 512>(p, TB, s));
  const bool one = p.T <= route_alone(p.E);
  if (e != hipSuccess || one) return e;
  const int64_t blocks = route_blocks(p.T, p.E);
  int cols = 4;  // threads of a row of the table
  while (4 * cols < route_row_bytes(p.E)) cols *= 2;
  const int threads = blocks * cols > 16 * 256 ? 1024 : 256;
  hipLaunchKernelGGL(route_place_kernel, dim3((unsigned)(blocks < 256 ? blocks : 256)), dim3(threads), 0, s, p, TB, (int)blocks, cols);
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
  if (p.top <= 16) {  // 16 lanes hold them
    if (p.E <= 64) return grad_launch<16, 4>(p, s);
    if (p.E <= 128) return grad_launch<16, 8>(p, s);
    if (p.E <= 256) return grad_launch<16, 16>(p, s);
  }
  if (p.E <= 256) return grad_launch<64, 4>(p, s);
  if (p.E <= 512) return grad_launch<64, 8>(p, s);
  return grad_launch<64, 16>(p, s);
}

}  // namespace tgemm
