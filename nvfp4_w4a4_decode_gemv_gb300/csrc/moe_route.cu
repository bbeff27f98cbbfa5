// Routing of tokens to experts: scores, the choice of the best, their weights,
// and the plan of the (token, expert) pairs by expert that the experts'
// products read.
//
// A warp takes a token; a lane holds NV experts that follow one another.  The choice is
// top_k rounds of a warp maximum over order-preserving integer keys (equal keys:
// the lowest expert).  Without a bias the keys are the logits themselves, since
// both scores grow with them: exact.  With a bias, or with groups ranked by the
// sum of two scores, the values are FP32 with a bound on their error; a token
// whose order that bound does not settle is chosen again from 64-bit values
// of the experts in question (one in some hundreds of tokens), so that the result
// is the one of the formulas in 64 bits.
//
// The plan is a stable counting sort: counts of a CTA's tokens by expert, sums
// over the CTAs before it, then ranks in the CTA by warp matches.  Every sum is of
// integers: no order of atomics shows.  Few tokens take one launch of one CTA;
// else the counts of a launch are what the second one begins with.
//
// Bound by latency, not by its bytes or its issue slots (a third of them are taken).  8 of 256 experts, 8192 tokens,
// sigmoid scores with a bias, 4 of 8 groups by their two best: 37 us (floor 1.4),
// some 7 of them the 64-bit values and 11 the plan; plain softmax 20 us.  One
// token of 128 experts: 4.5 us in a graph, 7 called from Python.
#include <math.h>

#include "common.cuh"

NVFP4_DEFINE_ERROR_READER(nvfp4_internal_read_error_moe_route)

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxExperts = 512;
constexpr int kMaxTop = 32;
constexpr int kMaxGroups = 32;
// Tokens that one CTA routes and plans by itself: one launch and no workspace (64 tokens, 6 of 64 experts in groups: 10.0 us
// called from Python, by two launches 14.1; in a graph 10.0 and 8.4; 32 tokens in a graph 6.1 and 6.3).
constexpr int kOneCta = 64;
constexpr int kMaxCtas = 152;             // of a call: bounds the workspace; one CTA an SM
constexpr uint32_t kAll = 0xFFFFFFFFu;

struct PlanArgs {
  int32_t *ids, *offsets, *pairs, *places;
  int32_t* counts;                        // [CTAs][experts], or NULL: one CTA does everything
  long long n_pairs;
  int experts, top, per;                  // per: tokens of a CTA
};

struct RouteArgs {
  PlanArgs plan;
  const void* logits;
  int64_t ld;
  const float* bias;
  const uint8_t* rows;
  float* weights;
  int tokens, groups, each, top_groups, group_best;
  uint32_t inv_each;                      // 2^20 / each, rounded up: expert * inv_each >> 20 is its group (expert < 512)
  int lanes;                              // of a group, where groups are whole lanes and a power of two of them; else 0
  int vector;                             // rows are read in 16-byte pieces
  int sigmoid, renormalize;
  float scale;
};

NVFP4_DEVINL float load1(const float* p) { return *p; }
NVFP4_DEVINL float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// Keys: unsigned integers in the order of the values; 0 is below every value's key.
NVFP4_DEVINL uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
NVFP4_DEVINL float value_of(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu)); }
NVFP4_DEVINL unsigned long long key_of(double v) {
  const unsigned long long b = (unsigned long long)__double_as_longlong(v);
  return b ^ ((b >> 63) ? ~0ull : 1ull << 63);
}
NVFP4_DEVINL double value_of(unsigned long long k) {
  return __longlong_as_double((long long)(k ^ ((k >> 63) ? 1ull << 63 : ~0ull)));
}
NVFP4_DEVINL uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kAll, k); }
NVFP4_DEVINL unsigned long long warp_max(unsigned long long k) {
  const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (unsigned long long)hi << 32 | lo;
}
template <class F> struct KeyOf;
template <> struct KeyOf<float> { using T = uint32_t; };
template <> struct KeyOf<double> { using T = unsigned long long; };

NVFP4_DEVINL float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
NVFP4_DEVINL double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// The largest key of the warp and the lowest lane that has it: lanes hold ascending experts.
template <class K>
NVFP4_DEVINL K warp_best(K best, int& lane_of) {
  const K m = warp_max(best);
  lane_of = __ffs(__ballot_sync(kAll, best == m)) - 1;
  return m;
}

// A lane's largest key and the first of its experts that has it.
template <class K, int NV>
NVFP4_DEVINL K lane_best(const K (&key)[NV], int& at) {
  K best = key[0];
  at = 0;
#pragma unroll
  for (int i = 1; i < NV; ++i)
    if (key[i] > best) {
      best = key[i];
      at = i;
    }
  return best;
}

// The two largest of (a0 >= a1) and (b0 >= b1).
template <class K>
NVFP4_DEVINL void merge_two(K& a0, K& a1, K b0, K b1) {
  const K lo = a0 < b0 ? a0 : b0, second = a1 > b1 ? a1 : b1;
  a0 = a0 > b0 ? a0 : b0;
  a1 = lo > second ? lo : second;
}
NVFP4_DEVINL uint32_t shfl_xor(uint32_t k, int o) { return __shfl_xor_sync(kAll, k, o); }
NVFP4_DEVINL unsigned long long shfl_xor(unsigned long long k, int o) { return __shfl_xor_sync(kAll, k, o); }

template <class K, int NV>
NVFP4_DEVINL void lane_two(const K (&key)[NV], K& first, K& second) {
  first = key[0];
  second = 0;
#pragma unroll
  for (int i = 1; i < NV; ++i) merge_two<K>(first, second, key[i], 0);
}

// Keys of a group's score: its largest value, or the sum of its two largest.
template <class F, class K>
NVFP4_DEVINL K group_score(const RouteArgs& a, K first, K second) {
  return a.group_best == 2 && a.each > 1 ? key_of(value_of(first) + value_of(second)) : first;
}

// Bit i: the group of this lane's expert i is one of the top_groups best by the sum of their group_best (1 or 2) largest
// values.  unsure: the first group left out is within 2 err of the last one kept.
template <class F, int NV>
NVFP4_DEVINL uint32_t kept_experts(const RouteArgs& a, const F (&v)[NV], int lane, F err, bool& unsure) {
  using K = typename KeyOf<F>::T;
  K key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) key[i] = lane * NV + i < a.plan.experts ? key_of(v[i]) : 0;
  K mine, last = 0;                          // the score of the lane's group, or of group `lane`
  uint32_t kept = 0u;
  if (a.lanes > 0) {
    // a group is `lanes` (a power of two) whole lanes: all groups at once
    K second;
    lane_two<K, NV>(key, mine, second);
    for (int o = 1; o < a.lanes; o <<= 1) merge_two<K>(mine, second, shfl_xor(mine, o), shfl_xor(second, o));
    mine = lane * NV < a.plan.experts ? group_score<F, K>(a, mine, second) : 0;
    for (int j = 0; j <= a.top_groups && j < a.groups; ++j) {
      int l;
      const K m = warp_best(mine, l);
      if (j == a.top_groups) {
        if (!(value_of(last) - value_of(m) > 2 * err)) unsure = true;
        break;
      }
      last = m;
      if (lane / a.lanes == l / a.lanes) {
        kept = kAll;
        mine = 0;
      }
    }
    return kept;
  }
  mine = 0;
  for (int g = 0; g < a.groups; ++g) {
    K in[NV], first, second;
#pragma unroll
    for (int i = 0; i < NV; ++i) in[i] = (int)(((uint32_t)(lane * NV + i) * a.inv_each) >> 20) == g ? key[i] : 0;
    lane_two<K, NV>(in, first, second);
    int owner;
    const K m1 = warp_best(first, owner);
    const K m2 = warp_max(lane == owner ? second : first);
    if (lane == g) mine = group_score<F, K>(a, m1, m2);
  }
  for (int j = 0; j <= a.top_groups && j < a.groups; ++j) {
    int g;
    const K m = warp_best(mine, g);
    if (j == a.top_groups) {
      if (!(value_of(last) - value_of(m) > 2 * err)) unsure = true;
      break;
    }
    last = m;
    if (lane == g) mine = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) kept |= (int)(((uint32_t)(lane * NV + i) * a.inv_each) >> 20) == g ? 1u << i : 0u;
  }
  return kept;
}

// Lane j's choice j (j < top_k) of the experts kept; c: what it goes by.  unsure: two neighbours in the order, the first left
// out among them, are within 2 err.  kth: the value of the last one chosen.
template <class F, int NV>
NVFP4_DEVINL int choose(const RouteArgs& a, const F (&c)[NV], uint32_t kept, int lane, F err, bool& unsure, F& kth) {
  using K = typename KeyOf<F>::T;
  K key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) key[i] = lane * NV + i < a.plan.experts && (kept >> i & 1u) ? key_of(c[i]) : 0;
  int at;
  K best = lane_best<K, NV>(key, at);
  int mine = -1;
  K last = 0;
  const int rounds = a.plan.top + (err > 0 ? 1 : 0);      // one more looks at the first that is left out
  for (int j = 0; j < rounds; ++j) {
    int owner;
    const K m = warp_best(best, owner);
    if (m == 0) break;                                    // nothing is left out
    if (j > 0 && err > 0 && !(value_of(last) - value_of(m) > 2 * err)) unsure = true;
    if (j < a.plan.top) last = m;
    const int i_of = __shfl_sync(kAll, at, owner);
    if (lane == j) mine = owner * NV + i_of;
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i == at) key[i] = 0;
      best = lane_best<K, NV>(key, at);
    }
  }
  kth = value_of(last);
  return mine;
}

// ---- the choice where FP32 does not settle it ------------------------------------------
// From 64-bit values of the experts that FP32 leaves in question, as a rule a handful.  A 64-bit exponential and quotient
// take a warp 2 us whether one lane needs them or all do: candidates are dealt out to the lanes, 32 at a time.
struct Scratch {                             // of a warp
  double value[32];
  int expert[32];
};

__device__ __noinline__ double score64(bool sigmoid, double x, double m, double z) {
  const double e = exp(sigmoid ? -x : x - m);
  return sigmoid ? 1.0 / (1.0 + e) : e / z;
}

// d[i] = the 64-bit value of each of this lane's experts i with bit i of `which` set.
template <int NV, class T>
NVFP4_DEVINL void exact_values(const RouteArgs& a, const T* row, Scratch& s, uint32_t which, double m, double z, int lane,
                               double (&d)[NV]) {
  const int n = __popc(which);
  int first = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kAll, first, o);
    if (lane >= o) first += x;
  }
  const int total = __shfl_sync(kAll, first, 31);
  first -= n;
#pragma unroll 1
  for (int at = 0; at < total; at += 32) {
    int k = first - at;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (which >> i & 1u) {
        if (k >= 0 && k < 32) s.expert[k] = lane * NV + i;
        ++k;
      }
    __syncwarp();
    if (at + lane < total) {
      const int e = s.expert[lane];
      const double v = score64(a.sigmoid != 0, (double)load1(row + e), m, z);
      s.value[lane] = a.bias ? v + (double)a.bias[e] : v;
    }
    __syncwarp();
    k = first - at;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (which >> i & 1u) {
        if (k >= 0 && k < 32) d[i] = s.value[k];
        ++k;
      }
    __syncwarp();
  }
}

// v: the FP32 values, off by err (groups: sums of two of them by v_err) at most.
template <int NV, class T>
__device__ __noinline__ int settle(const RouteArgs& a, const T* row, Scratch& s, const float* px, const float* pv, float m,
                                   float err, float v_err, int lane) {
  float x[NV], v[NV];
  double d[NV];
  uint32_t all = 0u;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    x[i] = px[i];
    v[i] = pv[i];
    d[i] = -INFINITY;
    all |= lane * NV + i < a.plan.experts ? 1u << i : 0u;
  }
  double z = 1.0;
  if (!a.sigmoid && a.bias) {                // (without a bias, scores of one token may do without their sum)
    z = 0.0;
#pragma unroll 1
    for (int i = 0; i < NV; ++i)
      if (all >> i & 1u) z += score64(false, (double)load1(row + lane * NV + i), m, 1.0);
    z = warp_sum(z);
  }
  uint32_t kept = kAll, known = 0u;
  bool unused = false;
  if (a.top_groups < a.groups) {
    known = all;                             // groups across lanes: all of them
    if (a.lanes > 0) {
      // of a group, what may be one of its group_best largest
      uint32_t key[NV], first, second;
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = all >> i & 1u ? key_of(v[i]) : 0u;
      lane_two<uint32_t, NV>(key, first, second);
      for (int o = 1; o < a.lanes; o <<= 1) merge_two<uint32_t>(first, second, shfl_xor(first, o), shfl_xor(second, o));
      const float least = value_of(a.group_best == 2 && a.each > 1 ? second : first);
      known = 0u;
#pragma unroll
      for (int i = 0; i < NV; ++i) known |= !(v[i] < least - 2.0f * v_err) ? 1u << i : 0u;
      known &= all;
    }
    exact_values<NV>(a, row, s, known, m, z, lane, d);
    kept = kept_experts<double, NV>(a, d, lane, 0.0, unused);
  }
  float kth;
  if (!a.bias) return choose<float, NV>(a, x, kept, lane, 0.0f, unused, kth);
  choose<float, NV>(a, v, kept, lane, 0.0f, unused, kth);
  uint32_t close = 0u;                       // what may be one of the chosen
#pragma unroll
  for (int i = 0; i < NV; ++i) close |= !(v[i] < kth - 2.0f * err) ? 1u << i : 0u;
  close &= kept & all;
  exact_values<NV>(a, row, s, close & ~known, m, z, lane, d);
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (!(close >> i & 1u)) d[i] = -INFINITY;
  double last;
  return choose<double, NV>(a, d, kept, lane, 0.0, unused, last);
}

// A lane's NV elements of a row, -inf beyond the experts; whole 16-byte pieces where the rows allow it.
template <int NV>
NVFP4_DEVINL void load_row(const RouteArgs& a, const float* row, int lane, float (&x)[NV]) {
  if constexpr (NV % 4 == 0) {
    if (a.vector && lane * NV + NV <= a.plan.experts) {
#pragma unroll
      for (int i = 0; i < NV / 4; ++i) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(row + lane * NV) + i);
        x[4 * i] = u.x, x[4 * i + 1] = u.y, x[4 * i + 2] = u.z, x[4 * i + 3] = u.w;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = lane * NV + i < a.plan.experts ? load1(row + lane * NV + i) : -INFINITY;
}
template <int NV>
NVFP4_DEVINL void load_row(const RouteArgs& a, const uint16_t* row, int lane, float (&x)[NV]) {
  if constexpr (NV % 8 == 0) {
    if (a.vector && lane * NV + NV <= a.plan.experts) {
#pragma unroll
      for (int i = 0; i < NV / 8; ++i) {
        const uint4 u = __ldcg(reinterpret_cast<const uint4*>(row + lane * NV) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) x[8 * i + 2 * j] = bf16_lo(w[j]), x[8 * i + 2 * j + 1] = bf16_hi(w[j]);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = lane * NV + i < a.plan.experts ? load1(row + lane * NV + i) : -INFINITY;
}

// One token by one warp: lane j < top_k returns its expert (-1: none) and writes it with its weight.
template <int NV, class T>
NVFP4_DEVINL int route_row(const RouteArgs& a, Scratch& scratch, int token, int lane) {
  const int E = a.plan.experts, top = a.plan.top;
  int id = -1;
  float w = 0.0f;
  if (!a.rows || a.rows[token] != 0) {
    const T* row = static_cast<const T*>(a.logits) + (size_t)token * a.ld;
    float x[NV], v[NV];
    float m = -INFINITY;
    bool bad = false;
    load_row<NV>(a, row, lane, x);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] += 0.0f;                                       // (both zeros are one value)
      bad = bad || isnan(x[i]);
      m = fmaxf(m, x[i]);
    }
    float z = 1.0f, c_err = 0.0f, v_err = 0.0f;
    if (!a.sigmoid) {
      m = value_of(warp_max(key_of(m)));
      bad = bad || isinf(m);
    }
    const bool sums = a.top_groups < a.groups && a.group_best == 2;
    if (a.bias || sums || (!a.sigmoid && !a.renormalize)) {
      // For the choice alone, with approximate exponentials and quotients, since their error is bounded and the weights
      // are computed again.
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        v[i] = a.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-x[i])) : __expf(x[i] - m);
        sum += v[i];
      }
      const float inv = a.sigmoid ? 1.0f : __fdividef(1.0f, warp_sum(sum));
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = lane * NV + i;
        v[i] *= inv;
        if (a.bias && e < E) {
          v[i] += a.bias[e];
          bad = bad || isnan(v[i]);
        }
        // (an infinite value settles nothing: the error is then infinite too)
        if (e < E) most = fmaxf(most, fabsf(v[i]));
      }
      most = __uint_as_float(warp_max(__float_as_uint(most)));
      // |v - exact| is below this.  __expf(t) is off by 2 + 1.173 |t| ulp, __fdividef by 2.  Sigmoid: e^-x is weighed with
      // s (1 - s), which makes at most 0.6 ulp of it; sum, quotient and bias add 3: 2^-21.  Softmax, each score at most
      // 1 / z = inv: (2 + 1.173 |t|) e^t is at most 2 ulp of the largest term, x - m loses half of one; z is off by 21
      // half ulps of up to 512 terms' sum and by 8.5 ulp of its terms' mean at worst (511 of them near t = -4.9 beside one at
      // 0, x - m rounded), the quotient by 2: 2^-18.4 of inv in all.  A sum of two values doubles it.  (e^-x that overflows
      // gives 0 and is off by 2^-126.)
      const float score = a.sigmoid ? 0x1p-20f : 0x1p-18f * fminf(1.0f, inv) + 0x1p-24f;
      v_err = 2.0f * (score + 0x1p-23f * most);
      if (a.bias) c_err = score + 0x1p-23f * most;
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = x[i];
    }
    if (!a.sigmoid && !a.renormalize) {
      float sum = 0.0f;                                   // for the weights
#pragma unroll
      for (int i = 0; i < NV; ++i) sum += expf(x[i] - m);
      z = warp_sum(sum);
    }
    bad = __any_sync(kAll, bad);
    if (!bad) {
      bool unsure = false;
      float kth;
      uint32_t kept = kAll;
      const bool by_value = a.bias || sums;
      if (a.top_groups < a.groups)
        kept = by_value ? kept_experts<float, NV>(a, v, lane, v_err, unsure) : kept_experts<float, NV>(a, x, lane, 0.0f, unsure);
      if (!by_value) unsure = false;                      // logits: equal ones are equal
      id = a.bias ? choose<float, NV>(a, v, kept, lane, c_err, unsure, kth)
                  : choose<float, NV>(a, x, kept, lane, 0.0f, unsure, kth);
      if (unsure) {
        float px[NV], pv[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) px[i] = x[i], pv[i] = v[i];
        id = settle<NV, T>(a, row, scratch, px, pv, m, c_err, v_err, lane);
      }
      const bool chosen = lane < top;
      const float xc = chosen ? load1(row + max(id, 0)) + 0.0f : -INFINITY;
      if (a.renormalize) {
        // exp(x) / (1 + exp(x)) and exp(x) alike, relative to the largest of the chosen: no sum underflows
        const float xm = value_of(warp_max(key_of(xc)));
        float t = 0.0f;
        if (chosen && xm > -INFINITY)
          t = a.sigmoid ? __fdiv_rn(expf(fminf(xc, 0.0f) - fminf(xm, 0.0f)), 1.0f + expf(-fabsf(xc))) : expf(xc - xm);
        const float sum = warp_sum(t);
        w = sum > 0.0f ? __fdiv_rn(t, sum) * a.scale : 0.0f;
      } else {
        w = (a.sigmoid ? __fdiv_rn(1.0f, 1.0f + expf(-xc)) : __fdiv_rn(expf(xc - m), z)) * a.scale;
      }
    } else if (lane == 0) {
      atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_NO_EXPERT);
    }
  }
  if (lane < top) {
    a.plan.ids[(size_t)token * top + lane] = id;
    a.weights[(size_t)token * top + lane] = w;
  }
  return lane < top ? id : -1;
}

// Exclusive sums of s_tot[0, n) over the first warp, into s_first[0, n]; n <= 512.
NVFP4_DEVINL void first_of_experts(const int* s_tot, int* s_first, int n) {
  const int lane = threadIdx.x, per = (n + 31) / 32;
  int sum = 0;
  for (int i = 0; i < per; ++i) sum += lane * per + i < n ? s_tot[lane * per + i] : 0;
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kAll, inc, o);
    if (lane >= o) inc += x;
  }
  int at = inc - sum;
  for (int i = 0; i < per; ++i)
    if (lane * per + i < n) {
      s_first[lane * per + i] = at;
      at += s_tot[lane * per + i];
    }
  if (lane == 31) s_first[n] = at;
}

// This CTA's pairs [p0, p1) to their places; ids: theirs from p0 on; s_next[e]: the next place of expert e; s_warp:
// kWarps * experts ints.
NVFP4_DEVINL void place_pairs(const PlanArgs& a, const int32_t* ids, long long p0, long long p1, int* s_next, int* s_warp) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, E = a.experts;
  for (long long p = p0; p < p1; p += kThreads) {
    const int warps = (int)((min(p1 - p, (long long)kThreads) + 31) / 32);   // that have pairs
    for (int i = tid; i < warps * E; i += kThreads) s_warp[i] = 0;
    __syncthreads();
    const long long pair = p + tid;
    int e = pair < p1 ? ids[pair - p0] : -1;
    if (e < 0 || e >= E) e = -1;
    const uint32_t same = __match_any_sync(kAll, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (e >= 0 && rank == 0) s_warp[warp * E + e] = __popc(same);
    __syncthreads();
    for (int i = tid; i < E; i += kThreads) {
      int at = s_next[i];
      for (int w = 0; w < warps; ++w) {
        const int n = s_warp[w * E + i];
        s_warp[w * E + i] = at;
        at += n;
      }
      s_next[i] = at;
    }
    __syncthreads();
    if (pair < p1) {
      const int at = e >= 0 ? s_warp[warp * E + e] + rank : -1;
      a.places[pair] = at;
      if (e >= 0) a.pairs[at] = (int)pair;
    }
    __syncthreads();
  }
}

// Entries of pairs behind the last one, this CTA's share.
NVFP4_DEVINL void fill_pairs(const PlanArgs& a, long long p0, long long p1, int total) {
  for (long long p = max(p0, (long long)total) + threadIdx.x; p < p1; p += kThreads) a.pairs[p] = -1;
}

extern __shared__ int s_dyn[];            // kWarps * experts, where a plan is made

// ids == NULL route; else (NV = 0): the ids are the caller's.
template <int NV, class T>
__global__ void __launch_bounds__(kThreads) moe_route_kernel(const RouteArgs a) {
  __shared__ int s_cnt[kMaxExperts], s_first[kMaxExperts + 1];
  __shared__ int32_t s_ids[kOneCta * kMaxTop];             // of the one CTA's tokens
  __shared__ Scratch s_scratch[NV > 0 ? kWarps : 1];
  const PlanArgs& pl = a.plan;
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < pl.experts; i += kThreads) s_cnt[i] = 0;
  __syncthreads();
  griddep_wait();
  const int t0 = min(blockIdx.x * pl.per, a.tokens), t1 = min(t0 + pl.per, a.tokens);
  const long long p0 = (long long)t0 * pl.top, p1 = (long long)t1 * pl.top;
  if constexpr (NV > 0) {
    for (int t = t0 + warp; t < t1; t += kWarps) {
      const int id = route_row<NV, T>(a, s_scratch[warp], t, lane);
      if (id >= 0) atomicAdd(&s_cnt[id], 1);
      if (!pl.counts && lane < pl.top) s_ids[t * pl.top + lane] = id;
    }
  } else {
    for (long long p = p0 + tid; p < p1; p += kThreads) {
      const int id = pl.ids[p];
      if (!pl.counts) s_ids[p] = id;
      if (id >= 0 && id < pl.experts) atomicAdd(&s_cnt[id], 1);
      else if (id != -1) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_MOE_RANGE);
    }
  }
  __syncthreads();
  if (pl.counts) {
    for (int i = tid; i < pl.experts; i += kThreads) pl.counts[(size_t)blockIdx.x * pl.experts + i] = s_cnt[i];
    return;
  }
  if (warp == 0) first_of_experts(s_cnt, s_first, pl.experts);
  __syncthreads();
  for (int i = tid; i <= pl.experts; i += kThreads) pl.offsets[i] = s_first[i];
  fill_pairs(pl, 0, pl.n_pairs, s_first[pl.experts]);
  __syncthreads();                        // s_first turns into the next places
  place_pairs(pl, s_ids, p0, p1, s_first, s_dyn);
}

__global__ void __launch_bounds__(kThreads) moe_place_kernel(const PlanArgs a) {
  __shared__ int s_tot[kMaxExperts], s_before[kMaxExperts], s_first[kMaxExperts + 1];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, E = a.experts, G = gridDim.x;
  for (int i = tid; i < E; i += kThreads) s_tot[i] = s_before[i] = 0;
  __syncthreads();
  const int parts = kThreads / E, part = tid / E, e = tid - part * E;
  if (part < parts) {
    int tot = 0, before = 0;
    const int b0 = part * G / parts, b1 = (part + 1) * G / parts;
#pragma unroll 8
    for (int b = b0; b < b1; ++b) {
      const int n = a.counts[(size_t)b * E + e];
      tot += n;
      if (b < (int)blockIdx.x) before += n;
    }
    atomicAdd(&s_tot[e], tot);
    atomicAdd(&s_before[e], before);
  }
  __syncthreads();
  if (tid < 32) first_of_experts(s_tot, s_first, E);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = tid; i <= E; i += kThreads) a.offsets[i] = s_first[i];
  const long long p0 = min((long long)blockIdx.x * a.per * a.top, a.n_pairs);
  const long long p1 = min(p0 + (long long)a.per * a.top, a.n_pairs);
  fill_pairs(a, p0, p1, s_first[E]);
  for (int i = tid; i < E; i += kThreads) s_tot[i] = s_first[i] + s_before[i];
  __syncthreads();
  place_pairs(a, a.ids + p0, p0, p1, s_tot, s_dyn);
}

template <class Args>
cudaError_t launch(void (*kern)(Args), int grid, size_t smem, const Args& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

using RouteKernel = void (*)(RouteArgs);

// Experts of a lane: the least that is built.
constexpr int kPerLane[] = {1, 2, 4, 5, 8, 12, 16};

int per_lane(int experts) {
  for (int nv : kPerLane)
    if (32 * nv >= experts) return nv;
  return 16;
}

template <class T>
RouteKernel kernel_for(int nv) {
  switch (nv) {
    case 1: return moe_route_kernel<1, T>;
    case 2: return moe_route_kernel<2, T>;
    case 4: return moe_route_kernel<4, T>;
    case 5: return moe_route_kernel<5, T>;
    case 8: return moe_route_kernel<8, T>;
    case 12: return moe_route_kernel<12, T>;
    default: return moe_route_kernel<16, T>;
  }
}

// The largest dynamic shared memory that a plan takes, allowed once a device for every kernel here.
cudaError_t allow_smem() {
  static PerDeviceInt done;
  cudaError_t err = cudaSuccess;
  done.get([](int, cudaError_t* e_out) -> int {
    const int bytes = kWarps * kMaxExperts * (int)sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(moe_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(moe_route_kernel<0, float>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    for (int nv : kPerLane)
      for (RouteKernel k : {kernel_for<float>(nv), kernel_for<uint16_t>(nv)})
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    *e_out = e;
    return e == cudaSuccess ? 1 : 0;
  }, &err);
  return err;
}

int ctas_for(int tokens) {
  if (tokens <= kOneCta) return 1;
  const int n = (tokens + kWarps - 1) / kWarps;
  return n < kMaxCtas ? n : kMaxCtas;
}

cudaError_t run(RouteKernel kern, RouteArgs a, cudaStream_t stream) {
  cudaError_t e = allow_smem();
  if (e != cudaSuccess) return e;
  const int ctas = ctas_for(a.tokens);
  a.plan.per = (a.tokens + ctas - 1) / ctas;
  a.plan.n_pairs = (long long)a.tokens * a.plan.top;
  const size_t smem = (size_t)kWarps * a.plan.experts * sizeof(int);
  if (ctas == 1) {
    a.plan.counts = nullptr;
    return launch(kern, 1, smem, a, stream);
  }
  e = launch(kern, ctas, 0, a, stream);
  return e == cudaSuccess ? launch(moe_place_kernel, ctas, smem, a.plan, stream) : e;
}

}  // namespace

nvfp4_status nvfp4_internal_cuda_status(cudaError_t e);
bool nvfp4_internal_aligned(const void* p, size_t a);
nvfp4_status nvfp4_internal_check_device();

namespace {

nvfp4_status check_plan(int tokens, int top_k, int experts, const PlanArgs& p, const void* workspace, size_t bytes) {
  if (experts < 1 || experts > kMaxExperts || tokens < 0 || top_k < 1 || top_k > kMaxTop) return NVFP4_ERR_SHAPE;
  if ((long long)tokens * top_k > 0x7FFFFFFFll) return NVFP4_ERR_SHAPE;
  if (!p.offsets || (tokens > 0 && (!p.ids || !p.pairs || !p.places))) return NVFP4_ERR_NULL;
  if (!nvfp4_internal_aligned(p.offsets, 4) || !nvfp4_internal_aligned(p.ids, 4) || !nvfp4_internal_aligned(p.pairs, 4) ||
      !nvfp4_internal_aligned(p.places, 4) || !nvfp4_internal_aligned(workspace, 4))
    return NVFP4_ERR_ALIGN;
  const size_t need = nvfp4_moe_route_workspace_bytes(tokens, experts);
  if (need > 0 && !workspace) return NVFP4_ERR_NULL;
  if (bytes < need) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

}  // namespace

extern "C" size_t nvfp4_moe_route_workspace_bytes(int tokens, int experts) {
  if (tokens < 0 || experts < 1 || experts > kMaxExperts) return 0;
  const int ctas = ctas_for(tokens);
  return ctas == 1 ? 0 : (size_t)ctas * experts * sizeof(int32_t);
}

extern "C" nvfp4_status nvfp4_moe_route(const void* logits, int dtype, int tokens, int experts, int64_t ld,
                                        const nvfp4_moe_router* r, const float* bias, const uint8_t* rows, int32_t* ids,
                                        float* weights, int32_t* offsets, int32_t* pairs, int32_t* places, void* workspace,
                                        size_t workspace_bytes, cudaStream_t stream) {
  if (!r) return NVFP4_ERR_NULL;
  RouteArgs a = {};
  a.plan.ids = ids, a.plan.offsets = offsets, a.plan.pairs = pairs, a.plan.places = places;
  a.plan.counts = static_cast<int32_t*>(workspace);
  const nvfp4_status cs = check_plan(tokens, r->top_k, experts, a.plan, workspace, workspace_bytes);
  if (cs != NVFP4_OK) return cs;
  if (r->groups < 1 || r->groups > kMaxGroups || experts % r->groups != 0 || r->top_groups < 1 ||
      r->top_groups > r->groups || r->top_k > experts / r->groups * r->top_groups || ld < experts)
    return NVFP4_ERR_SHAPE;
  if (dtype != NVFP4_DTYPE_F32 && dtype != NVFP4_DTYPE_BF16) return NVFP4_ERR_RANGE;
  if (r->score != NVFP4_MOE_SOFTMAX && r->score != NVFP4_MOE_SIGMOID) return NVFP4_ERR_RANGE;
  if (r->group_best < 1 || r->group_best > 2 || !isfinite(r->scale)) return NVFP4_ERR_RANGE;
  if (tokens > 0 && (!logits || !weights)) return NVFP4_ERR_NULL;
  if (!nvfp4_internal_aligned(logits, dtype == NVFP4_DTYPE_F32 ? 4 : 2) || !nvfp4_internal_aligned(bias, 4) ||
      !nvfp4_internal_aligned(weights, 4))
    return NVFP4_ERR_ALIGN;
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  a.plan.experts = experts, a.plan.top = r->top_k;
  a.logits = logits, a.ld = ld, a.bias = bias, a.rows = rows, a.weights = weights;
  a.tokens = tokens, a.groups = r->groups, a.each = experts / r->groups, a.top_groups = r->top_groups;
  a.group_best = r->group_best, a.sigmoid = r->score == NVFP4_MOE_SIGMOID, a.renormalize = r->renormalize != 0;
  a.scale = r->scale;
  a.inv_each = ((1u << 20) + a.each - 1) / a.each;
  const int nv = per_lane(experts), lanes = a.each % nv == 0 ? a.each / nv : 0;
  a.lanes = lanes > 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  const int per = dtype == NVFP4_DTYPE_F32 ? 4 : 8;          // elements of 16 bytes
  a.vector = nvfp4_internal_aligned(logits, 16) && (tokens < 2 || ld % per == 0);
  return nvfp4_internal_cuda_status(run(dtype == NVFP4_DTYPE_F32 ? kernel_for<float>(nv) : kernel_for<uint16_t>(nv), a, stream));
}

extern "C" nvfp4_status nvfp4_moe_plan(const int32_t* ids, int tokens, int top_k, int experts, int32_t* offsets,
                                       int32_t* pairs, int32_t* places, void* workspace, size_t workspace_bytes,
                                       cudaStream_t stream) {
  RouteArgs a = {};
  a.plan.ids = const_cast<int32_t*>(ids), a.plan.offsets = offsets, a.plan.pairs = pairs, a.plan.places = places;
  a.plan.counts = static_cast<int32_t*>(workspace);
  const nvfp4_status cs = check_plan(tokens, top_k, experts, a.plan, workspace, workspace_bytes);
  if (cs != NVFP4_OK) return cs;
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  a.plan.experts = experts, a.plan.top = top_k;
  a.tokens = tokens;
  return nvfp4_internal_cuda_status(run(moe_route_kernel<0, float>, a, stream));
}
