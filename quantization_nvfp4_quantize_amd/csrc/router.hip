// Routing of tokens to experts on gfx950: expert ids and weights from the
// router's logits, in the form the expert FFN takes them.
//
// Per token, with logits z_e (NaN and -inf: the expert is masked; +inf counts
// as the largest finite value):
//   score   s_e = exp(z_e - max z) / sum exp(z - max z)   or   1 / (1 + exp(-z_e))
//   choice  c_e = s_e + bias_e; without a bias the order of z_e, which is the
//           order of s_e and needs no exponential
//   groups  of E / n_group consecutive experts; a group's value is the sum of
//           its group_top (1 or 2) largest choices; the topk_group best stay
//   ids     the k largest choices of the groups that stay, descending
//   weight  scale * s_e, or scale * s_e / (sum of the k chosen scores)
// Ties go to the lowest index.  The order is that of the values above in fp64,
// where those that fp64 cannot separate (sigmoids of logits beyond 37, softmax
// terms that underflow, scores that a bias swallows) tie.  Scores in fp32 carry
// errors of up to some 30 * 2^-24, so a decision between two values closer than
// a bound on those errors (at kGap) is taken again in fp64, for the whole
// token.  How many tokens that takes depends on the data, equal values among
// them: 16384 tokens of 256 experts with biases in steps of 0.001 take 20 to 22
// us whatever the logits; with equal biases bf16 logits, many of them equal,
// take 29 to 30, and softmax scores of logits spread by 0.02, all within the
// bound, 35.
//
// One wave holds one token; lane l the v experts g S + (l % Lg) v + 0 .. v-1
// of group g = l / Lg, with Lg = 64 / (n_group rounded up to a power of two)
// lanes per group.  A lane then has experts of one group only, so a group's
// value is a butterfly over Lg lanes and dropping a group clears whole lanes;
// and lower lanes hold lower experts, so the first lane of a ballot is the
// lowest index.  Each lane sorts its v values once; a pick is a wave maximum of
// the lanes' heads (six DPP maxima), a ballot, and a pop in the winning lane.
//
// Bound by the vector ALU for many tokens: 629 instructions per token with 8
// groups and a bias, 351 without, k 8; 16384 tokens of 256 experts take 22.5 and
// 10.8 us, where their 17 MB take 3.6.  One token: 4.5 us.
#include <hip/hip_runtime.h>

#include <float.h>

#include "launch.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

namespace {

constexpr int kRouteRows = 4;  // tokens (waves) per workgroup

struct RouteParams {
  const void* logits;       // [T][E] bf16 or fp32
  const float* bias;        // nullable [E]
  const int32_t* n_tokens;  // nullable: tokens that count; the rest get id -1, weight 0
  int64_t T;
  int E, k;
  int S, v;                 // experts per group, experts per lane
  int lanes_log2;           // log2 of the lanes per group
  int n_group, topk_group, group_top;
  int renormalize;
  float scale;
  int32_t* ids;             // [T][k]
  float* w;                 // [T][k]
};

// Order-preserving map of a float (never NaN) to an unsigned key; 0 is below
// every value and stands for a masked or taken expert.
__device__ __forceinline__ uint32_t key_of(float c) {
  const uint32_t b = __float_as_uint(c);
  return b ^ ((b & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key ^ ((key & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp0(uint32_t x) {  // lanes without a source read 0
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp_self(float x) {
  const int v = __float_as_int(x);
  return __int_as_float(__builtin_amdgcn_update_dpp(v, v, CTRL, 0xf, 0xf, false));
}
constexpr int kRowShr1 = 0x111, kRowShr2 = 0x112, kRowShr4 = 0x114, kRowShr8 = 0x118;
constexpr int kRowBcast15 = 0x142, kRowBcast31 = 0x143;
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

// Largest key of the wave, in every lane.  (Rows that a broadcast reaches
// twice see a value again, which a maximum does not mind.)
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = max(x, dpp0<kRowShr1>(x));
  x = max(x, dpp0<kRowShr2>(x));
  x = max(x, dpp0<kRowShr4>(x));
  x = max(x, dpp0<kRowShr8>(x));
  x = max(x, dpp0<kRowBcast15>(x));
  x = max(x, dpp0<kRowBcast31>(x));
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

// Swap within 2^(step+1) lanes, for values that are equal inside 2^step lanes
// (so a mirror is as good as an exchange).
template <class F>
__device__ __forceinline__ F swap_step(F x, int step);
template <>
__device__ __forceinline__ float swap_step<float>(float x, int step) {
  switch (step) {
    case 0: return dpp_self<kQuadXor1>(x);
    case 1: return dpp_self<kQuadXor2>(x);
    case 2: return dpp_self<kHalfMirror>(x);
    case 3: return dpp_self<kMirror>(x);
    case 4: return __shfl_xor(x, 16);
    default: return __shfl_xor(x, 32);
  }
}
template <>
__device__ __forceinline__ double swap_step<double>(double x, int step) {
  return __shfl_xor(x, 1 << step);
}

template <class F>
__device__ __forceinline__ F wave_max_f(F x) {
#pragma unroll
  for (int s = 0; s < 6; ++s) {
    const F y = swap_step(x, s);
    x = y > x ? y : x;
  }
  return x;
}
template <class F>
__device__ __forceinline__ F wave_sum(F x) {
#pragma unroll
  for (int s = 0; s < 6; ++s) x += swap_step(x, s);
  return x;
}

// The fp32 forms serve decisions only, whose margins cover their errors: the
// hardware's exp2 of a rounded product (relative error |x| 1.44 * 2^-24 + 2^-23)
// and its reciprocal (2^-23).
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
// exp for the weights: the product's rounding is given back (the hardware's
// exp2 and a half step or two remain); results below 2^-126 become 0.
__device__ __forceinline__ float weight_exp(float x) {
  const float hi = 1.44269502f, lo = 1.92596300e-8f;  // log2(e)
  const float t = x * hi, e = __builtin_amdgcn_exp2f(t);
  const float rest = __builtin_fmaf(x, lo, __builtin_fmaf(x, hi, -t));
  return e > 0.0f && e < INFINITY ? __builtin_fmaf(e, rest * 0.693147181f, e) : e;
}
__device__ __forceinline__ float inverse(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ double inverse(double x) { return 1.0 / x; }
__device__ __forceinline__ double lane_of(double x, int lane) {
  const long long b = __double_as_longlong(x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// A reduction over the first k lanes (at most 32; the others hold values that
// change nothing), in those lanes.
template <class Op>
__device__ __forceinline__ float first_lanes(float x, int k, Op op) {
#pragma unroll
  for (int s = 0; s < 4; ++s) x = op(x, swap_step(x, s));
  return k > 16 ? op(x, swap_step(x, 4)) : x;
}

// The gap up to which two choices c = s + bias may be in the wrong order in fp32,
// in units of u = 2^-24, the largest relative error of one rounding.
// Softmax, x = z - mx: a numerator exp(x) is off by (2.25 |x| + 2) u (difference,
// product with a rounded constant, exp2); the sum by that of its terms in the
// mean plus 20 u (14 additions of a lane's at most 15 experts, 6 of the lanes),
// its reciprocal by 2 u, the product by u.  Sum and reciprocal move all scores of
// a token by one factor, so the difference of two is off by
//   |s1 - s2| (24 + 2.25 sum_e s_e |x_e|) u + s1 (2.25 |x1| + 3) u + s2 (2.25 |x2| + 3) u,
// at most 27.1 u over all scores that add up to 1, and below 32 u for the sums of
// two scores of two groups.  Sigmoid: s (1 - s) (2.25 |z| + 2) u + 3 u < 5 u per
// score.  Then |c| u for each choice's own rounding: 32 u + 4 |c| u covers two
// choices, twice that two sums of two, which are rounded themselves.
constexpr float kGap = 0x1p-19f, kGapBias = 0x1p-22f;

// Scores of a lane's experts (0 for masked ones); mx, sum: the softmax's
// maximum and sum over the token (all lanes).
template <int V, bool SIGMOID, class F>
__device__ __forceinline__ void scores(const float (&z)[V], float mx, F& sum, F (&s)[V]) {
  F part = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const bool live = z[j] > -INFINITY;
    if (SIGMOID) {
      s[j] = live ? inverse((F)1 + exp_of(-(F)z[j])) : (F)0;
    } else {
      s[j] = live ? exp_of((F)z[j] - (F)mx) : (F)0;
      part += s[j];
    }
  }
  if (!SIGMOID) {
    sum = wave_sum(part);
    const F inv = sum > 0 ? inverse(sum) : (F)0;
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] *= inv;
  }
}

// Value of this lane's group: the sum of the one or two largest of its experts'
// values, -inf for a group with nothing.  In fp32 from keys (0: masked), whose
// maxima and minima are single instructions, across lanes too.
template <int CTRL>
__device__ __forceinline__ void merge2(uint32_t& a, uint32_t& b) {
  const uint32_t a2 = dpp0<CTRL>(a), b2 = dpp0<CTRL>(b);
  b = max(max(b, b2), min(a, a2));
  a = max(a, a2);
}
template <int V>
__device__ __forceinline__ float group_value(const RouteParams& p, const uint32_t (&k)[V]) {
  uint32_t a = k[0], b = 0u;
#pragma unroll
  for (int j = 1; j < V; ++j) {
    b = max(b, min(k[j], a));
    a = max(a, k[j]);
  }
  const int n = p.lanes_log2;
  if (n > 0) merge2<kQuadXor1>(a, b);
  if (n > 1) merge2<kQuadXor2>(a, b);
  if (n > 2) merge2<kHalfMirror>(a, b);
  if (n > 3) merge2<kMirror>(a, b);
  for (int s = 16; s < 1 << n; s <<= 1) {
    const uint32_t a2 = (uint32_t)__shfl_xor((int)a, s), b2 = (uint32_t)__shfl_xor((int)b, s);
    b = max(max(b, b2), min(a, a2));
    a = max(a, a2);
  }
  return !a ? -INFINITY : p.group_top == 2 && b ? value_of(a) + value_of(b) : value_of(a);
}
template <int V>
__device__ __forceinline__ double group_value(const RouteParams& p, const double (&g)[V]) {
  double a = g[0], b = -INFINITY;
#pragma unroll
  for (int j = 1; j < V; ++j) {
    const double lo = g[j] < a ? g[j] : a;
    a = g[j] > a ? g[j] : a;
    b = lo > b ? lo : b;
  }
  for (int s = 1; s < 1 << p.lanes_log2; s <<= 1) {
    const double a2 = __shfl_xor(a, s), b2 = __shfl_xor(b, s);
    const double lo = a2 < a ? a2 : a, b3 = b2 > b ? b2 : b;
    a = a2 > a ? a2 : a;
    b = lo > b3 ? lo : b3;
  }
  return p.group_top == 2 && b > -INFINITY ? a + b : a;
}

// Whether this lane's group is among the topk_group best (ties: the lowest
// group, so that a lower group is ahead with an equal value).
__device__ __forceinline__ bool keep_group(const RouteParams& p, float value, int group) {
  const uint32_t own = key_of(value + 0.0f);  // never 0: value >= -inf
  int ahead = 0;
  for (int g = 0; g < p.n_group; ++g) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)own, g << p.lanes_log2);
    ahead += o > (g < group ? own - 1 : own);
  }
  return ahead < p.topk_group;
}
__device__ __forceinline__ bool keep_group(const RouteParams& p, double value, int group) {
  int ahead = 0;
  for (int g = 0; g < p.n_group; ++g) {
    const double o = lane_of(value, g << p.lanes_log2);
    ahead += o > value || (o == value && g < group);
  }
  return ahead < p.topk_group;
}

template <int V, bool BF16, bool VEC>
__device__ __forceinline__ void load_logits(const RouteParams& p, int64_t t, int e0, int n, float (&z)[V]) {
  if (BF16) {
    const uint16_t* src = static_cast<const uint16_t*>(p.logits) + t * p.E + e0;
    if constexpr (VEC && V == 2) {
      if (n) {
        const uint32_t q = *reinterpret_cast<const uint32_t*>(src);
        z[0] = bf16_lo(q);
        z[1] = bf16_hi(q);
      }
    } else if constexpr (VEC && V == 4) {
      if (n) {
        const uint2 q = *reinterpret_cast<const uint2*>(src);
        z[0] = bf16_lo(q.x);
        z[1] = bf16_hi(q.x);
        z[2] = bf16_lo(q.y);
        z[3] = bf16_hi(q.y);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j < n) z[j] = bf16_lo(src[j]);
    }
  } else {
    const float* src = static_cast<const float*>(p.logits) + t * p.E + e0;
    if constexpr (VEC && V == 2) {
      if (n) {
        const float2 q = *reinterpret_cast<const float2*>(src);
        z[0] = q.x;
        z[1] = q.y;
      }
    } else if constexpr (VEC && V == 4) {
      if (n) {
        const float4 q = *reinterpret_cast<const float4*>(src);
        z[0] = q.x;
        z[1] = q.y;
        z[2] = q.z;
        z[3] = q.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j < n) z[j] = src[j];
    }
  }
}

// A logit as the routing sees it: -inf for masked, no +inf, no -0.
__device__ __forceinline__ float clean(float z) { return z > -INFINITY ? fminf(z, FLT_MAX) + 0.0f : -INFINITY; }

template <int V, bool BF16, bool SIGMOID, bool VEC>
__global__ __launch_bounds__(64 * kRouteRows) void moe_route_kernel(RouteParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kRouteRows + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= p.T) return;
  if (p.n_tokens && t >= *p.n_tokens) {
    if (lane < p.k) {
      p.ids[t * p.k + lane] = -1;
      p.w[t * p.k + lane] = 0.0f;
    }
    return;
  }
  const int group = lane >> p.lanes_log2;
  const int in_group = (lane & ((1 << p.lanes_log2) - 1)) * p.v;  // first expert of the lane within its group
  const int e0 = group * p.S + in_group;
  const int n = group < p.n_group ? max(0, min(p.v, p.S - in_group)) : 0;
  float z[V];
#pragma unroll
  for (int j = 0; j < V; ++j) z[j] = -INFINITY;
  load_logits<V, BF16, VEC>(p, t, e0, n, z);
#pragma unroll
  for (int j = 0; j < V; ++j) z[j] = clean(z[j]);

  const bool grouped = p.n_group > 1;
  const bool by_score = p.bias || (grouped && p.group_top == 2);  // some decision needs the scores
  float mx = 0.0f, sum = 1.0f, s[V];
  if (!SIGMOID && (by_score || !p.renormalize)) {
    float m = z[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, z[j]);
    mx = wave_max_f(m);
    if (!(mx > -INFINITY)) mx = 0.0f;
  }
  if (by_score || (!SIGMOID && !p.renormalize)) scores<V, SIGMOID>(z, mx, sum, s);

  int my_e = -1;     // lane i: the i-th expert
  bool unsure = false;
  {
    uint32_t key[V];
    int idx[V];
    float bias[V];
    if (p.bias) {
#pragma unroll
      for (int j = 0; j < V; ++j) bias[j] = j < n ? p.bias[e0 + j] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float c = p.bias ? (z[j] > -INFINITY ? s[j] + bias[j] + 0.0f : -INFINITY) : z[j];
      key[j] = c > -INFINITY ? key_of(c) : 0u;
      idx[j] = e0 + j;
    }
    if (grouped) {
      uint32_t g[V];
#pragma unroll
      for (int j = 0; j < V; ++j) g[j] = key[j] && by_score && !p.bias ? key_of(s[j]) : key[j];
      const float value = group_value(p, g);
      const bool keep = keep_group(p, value, group);
      if (by_score) {
        // the worst group that stays against the best that goes: two sums of
        // two choices; equal or infinite values count as close.  Scores are at
        // most 1; with a bias the largest |c| bounds the errors (a sum may be
        // small where its terms are not).
        const bool in = group < p.n_group;
        const uint32_t kv = key_of(value);
        const uint32_t low = ~wave_max(in && keep ? ~kv : 0u), high = wave_max(in && !keep ? kv : 0u);
        float most = 1.0f;
        if (p.bias) {
          uint32_t m = 0u;
#pragma unroll
          for (int j = 0; j < V; ++j) m = max(m, key[j] ? __float_as_uint(value_of(key[j])) & 0x7fffffffu : 0u);
          most = __uint_as_float(wave_max(m));
        }
        unsure = high != 0u && !(value_of(low) - value_of(high) > 2.0f * kGap + 2.0f * kGapBias * most);
      }
      if (!keep) {
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = 0u;
      }
    }
    // each lane's experts, largest key first, equal keys by index
    // (exchanges of neighbours only, so equal keys keep their order)
#pragma unroll
    for (int a = 0; a < V - 1; ++a) {
#pragma unroll
      for (int b = V - 2; b >= a; --b) {
        // on copies: a conditional between array elements selects an address,
        // which costs 13 instructions here instead of 5
        const uint32_t k0 = key[b], k1 = key[b + 1];
        const int i0 = idx[b], i1 = idx[b + 1];
        const bool sw = k1 > k0;
        key[b] = max(k0, k1);
        key[b + 1] = min(k0, k1);
        idx[b] = sw ? i1 : i0;
        idx[b + 1] = sw ? i0 : i1;
      }
    }
    const int picks = p.bias ? p.k + 1 : p.k;  // one more tells how near the next expert came
    uint32_t my_key = 0u;  // lane i: the key of the i-th pick
    int n_picked = 0;
    for (; n_picked < picks; ++n_picked) {
      const uint32_t best = wave_max(key[0]);
      if (best == 0) break;
      const int win = __ffsll((unsigned long long)__ballot(key[0] == best)) - 1;
      const int e = __builtin_amdgcn_readlane(idx[0], win);
      if (lane == n_picked) {
        my_e = e;
        my_key = best;
      }
      if (lane == win) {
#pragma unroll
        for (int j = 0; j < V - 1; ++j) {
          key[j] = key[j + 1];
          idx[j] = idx[j + 1];
        }
        key[V - 1] = 0u;
      }
    }
    if (p.bias) {
      // every pick against the next; a NaN gap (inf - inf) counts as close
      const uint32_t next_key = (uint32_t)__shfl_down((int)my_key, 1);
      const float c = value_of(my_key), next = value_of(next_key);
      unsure = unsure || __ballot(lane + 1 < n_picked && !(c - next > kGap + kGapBias * fabsf(next))) != 0;
    }
    if (lane >= p.k) my_e = -1;
  }

  if (__builtin_amdgcn_readfirstlane((int)unsure)) {
    // the same decisions in fp64
    double sd[V], sumd = 1.0, c[V];
    scores<V, SIGMOID>(z, mx, sumd, sd);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const double cj = p.bias ? sd[j] + (double)(j < n ? p.bias[e0 + j] : 0.0f) : (double)z[j];
      c[j] = z[j] > -INFINITY && cj > -INFINITY ? cj : -INFINITY;
    }
    bool open = true;
    if (grouped) {
      double g[V];
#pragma unroll
      for (int j = 0; j < V; ++j) g[j] = c[j] > -INFINITY ? (by_score && !p.bias ? sd[j] : c[j]) : -INFINITY;
      open = keep_group(p, group_value(p, g), group);
    }
    my_e = -1;
    uint32_t taken = 0;
    for (int i = 0; i < p.k; ++i) {
      double best = -INFINITY;
      int at = -1;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (open && !((taken >> j) & 1u) && c[j] > best) {
          best = c[j];
          at = j;
        }
      }
      const double top = wave_max_f(best);
      if (!(top > -INFINITY)) break;
      const int win = __ffsll((unsigned long long)__ballot(at >= 0 && best == top)) - 1;
      const int e = __builtin_amdgcn_readlane(e0 + at, win);
      my_e = lane == i ? e : my_e;
      if (lane == win) taken |= 1u << at;
    }
  }

  // weights: lane i has the i-th expert
  float zi = -INFINITY;
  if (my_e >= 0)
    zi = clean(BF16 ? bf16_lo(static_cast<const uint16_t*>(p.logits)[t * p.E + my_e])
                    : static_cast<const float*>(p.logits)[t * p.E + my_e]);
  float w;
  if (p.renormalize) {
    // every score over e^m, so that a token whose scores are all tiny keeps
    // their ratios: m = the largest chosen logit (softmax), or that where it
    // is negative (sigmoid).  Without a bias the first pick has it.
    float peak = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(zi)));
    if (p.bias) peak = first_lanes(zi, p.k, [](float x, float y) { return y > x ? y : x; });
    float part = 0.0f;
    if (my_e >= 0) {
      if (SIGMOID) {
        const float m = fminf(peak, 0.0f);
        part = zi > 0.0f ? inverse(1.0f + weight_exp(-zi)) : weight_exp(zi - m) * inverse(1.0f + weight_exp(zi));
      } else {
        part = weight_exp(zi - peak);
      }
    }
    const float total = first_lanes(part, p.k, [](float x, float y) { return x + y; });
    w = my_e >= 0 ? part * inverse(total) * p.scale : 0.0f;
  } else if (SIGMOID) {
    w = my_e >= 0 ? p.scale * inverse(1.0f + weight_exp(-zi)) : 0.0f;
  } else {
    w = my_e >= 0 ? weight_exp(zi - mx) * inverse(sum) * p.scale : 0.0f;
  }
  if (lane < p.k) {
    p.ids[t * p.k + lane] = my_e;
    p.w[t * p.k + lane] = w;
  }
}

template <int V, bool VEC>
hipError_t route_go(const RouteParams& p, bool bf16, bool sigmoid, hipStream_t s) {
  const dim3 grid((unsigned)((p.T + kRouteRows - 1) / kRouteRows)), block(64 * kRouteRows);
  if (bf16)
    sigmoid ? moe_route_kernel<V, true, true, VEC><<<grid, block, 0, s>>>(p)
            : moe_route_kernel<V, true, false, VEC><<<grid, block, 0, s>>>(p);
  else
    sigmoid ? moe_route_kernel<V, false, true, VEC><<<grid, block, 0, s>>>(p)
            : moe_route_kernel<V, false, false, VEC><<<grid, block, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_route(const void* logits, bool bf16, int64_t T, int E, const float* bias, bool sigmoid, int k,
                            int n_group, int topk_group, int group_top, bool renormalize, float scale,
                            const int32_t* n_tokens, int32_t* ids, float* w, hipStream_t s) {
  RouteParams p;
  p.logits = logits;
  p.bias = bias;
  p.n_tokens = n_tokens;
  p.T = T;
  p.E = E;
  p.k = k;
  p.S = E / n_group;
  int groups_log2 = 0;
  while ((1 << groups_log2) < n_group) ++groups_log2;
  p.lanes_log2 = 6 - groups_log2;
  const int lanes = 1 << p.lanes_log2;
  p.v = (p.S + lanes - 1) / lanes;
  p.n_group = n_group;
  p.topk_group = topk_group;
  p.group_top = group_top;
  p.renormalize = renormalize;
  p.scale = scale;
  p.ids = ids;
  p.w = w;
  // whole-lane vector loads: every lane's v experts are there and aligned
  if (p.v > 16) return hipErrorInvalidValue;  // never for n_group <= 64 and E <= 512
  const bool vec = p.S % p.v == 0 && E % p.v == 0 && (p.v == 2 || p.v == 4);
  if (p.v == 1) return route_go<1, false>(p, bf16, sigmoid, s);
  if (p.v == 2) return vec ? route_go<2, true>(p, bf16, sigmoid, s) : route_go<2, false>(p, bf16, sigmoid, s);
  if (p.v <= 4) return vec ? route_go<4, true>(p, bf16, sigmoid, s) : route_go<4, false>(p, bf16, sigmoid, s);
  if (p.v <= 8) return route_go<8, false>(p, bf16, sigmoid, s);
  return route_go<16, false>(p, bf16, sigmoid, s);
}

}  // namespace nvfp4
