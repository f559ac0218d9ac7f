// The router of a mixture-of-experts layer and its gradient: one warp per token.
//
// Scores are s = softmax(l) or sigmoid(l); the choice goes by key = s + bias.  Without a bias
// the keys are the logits themselves (both scores grow with the logit): the comparison is
// exact.  With one, 32-bit keys carry the rounding of the exponential, the division, the sum
// and the addition; where two neighbours in the chosen order (or the last chosen and the
// first left out, or two groups' ranks) are closer than a bound on that error, the token's
// selection is done again with 64-bit scores, of the experts that come into question only.
//
// route_kernel (up to 256 experts, groups of whole lanes): a lane holds V neighbouring
// experts as unsigned keys whose low bits are the place in the lane, sorted by a network of
// min/max; a step of the selection is then one reduction of the lanes' heads, one vote and a
// shift in the winning lane.  route_any_kernel takes any count and grouping: experts lane,
// lane + 32, ..., and a pass over the lane's registers at every step.  32768 tokens x 256
// experts, 8 chosen out of 4 of 8 groups: 36.4 us against 139 us.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "moe_launch.h"
#include "moe_ptx.cuh"

namespace cusync {
namespace moe {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Over groups of N neighbouring lanes (32: the warp).
template <int N = 32>
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = N / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
template <int N = 32>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = N / 2; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Bits that compare as unsigned integers as the floats do; both zeros alike.
__device__ __forceinline__ uint32_t ordered(float f) {
  const int32_t u = __float_as_int(f + 0.0f);
  return (uint32_t)u ^ ((uint32_t)(u >> 31) | 0x80000000u);
}

// The warp's largest (key, lowest index); index INT_MAX where every key is -inf.
__device__ __forceinline__ void warp_best(float& key, int& idx) {
  const uint32_t o = ordered(key);
  const uint32_t m = __reduce_max_sync(kFull, o);
  idx = (int)__reduce_min_sync(kFull, o == m ? (unsigned)idx : 0x7fffffffu);
  key = __uint_as_float((m & 0x80000000u) ? (m & 0x7fffffffu) : ~m);
}
__device__ __forceinline__ void warp_best(double& key, int& idx) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const double k2 = __shfl_xor_sync(kFull, key, o);
    const int i2 = __shfl_xor_sync(kFull, idx, o);
    if (k2 > key || (k2 == key && i2 < idx)) {
      key = k2;
      idx = i2;
    }
  }
}

// l - most for softmax's exponential; a logit of +inf is as far from the largest as what it tends
// to, 0 from itself and from others of its kind.
template <typename F>
__device__ __forceinline__ F below(F l, F most) {
  return l == most ? (F)0 : l - most;
}

// The rank of a group by its two largest keys: -inf where there is no second one, also beside
// a first of +inf (whose sum is a NaN, which the maximum drops).
__device__ __forceinline__ float rank_of_two(float first, float second) { return fmaxf(first + second, -INFINITY); }
__device__ __forceinline__ double rank_of_two(double first, double second) { return fmax(first + second, (double)-INFINITY); }

// Keeps the keys of the group_limit best groups, sets the others to -inf.  A group's rank
// is the sum of its group_top (1 or 2) largest keys.  Lane g ends with group g's rank.
// Returns false if ranks that decide are closer than tol.
template <typename F, int V>
__device__ bool keep_groups(const RouteArgs& a, F (&key)[V], int lane, F tol) {
  const F none = -(F)INFINITY;
  F rank = none;
  for (int g = 0; g < a.groups; ++g) {
    const int lo = g * a.group_size, hi = lo + a.group_size;
    F b1 = none;
    int i1 = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 32 * i;
      if (e >= lo && e < hi && key[i] > b1) {
        b1 = key[i];
        i1 = e;
      }
    }
    F m1 = b1;
    int j1 = i1;
    warp_best(m1, j1);
    F r = m1;
    if (a.group_top == 2 && a.group_size > 1) {
      F b2 = none;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        if (e >= lo && e < hi && e != j1 && key[i] > b2) b2 = key[i];
      }
      int j2 = 0x7fffffff;
      warp_best(b2, j2);
      r = rank_of_two(m1, b2);
    }
    if (lane == g) rank = r;
  }
  // the groups in order of rank: group_limit rounds, the last of them against the next best
  unsigned kept = 0;
  bool sure = true;
  F left = lane < a.groups ? rank : none;
  bool taken = lane >= a.groups;
  F last = none;
  for (int n = 0; n <= a.group_limit && n < a.groups; ++n) {
    // among equal ranks (-inf ones too) the lowest untaken group
    F best = taken ? none : left;
    int who = taken ? 0x7fffffff : lane;
    warp_best(best, who);
    if (n == a.group_limit) {
      if (last != none && !(last - best > tol)) sure = false;
      break;
    }
    kept |= 1u << who;
    if (lane == who) taken = true;
    last = best;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    if (e < a.E && !((kept >> (e / a.group_size)) & 1u)) key[i] = none;
  }
  return sure;
}

// The k best keys: lane j ends with the j-th one's expert (-1: none left).  Returns false
// if two neighbours of the order, or the last one and the first left out, are closer than
// tol.
template <typename F, int V>
__device__ bool pick(const RouteArgs& a, F (&key)[V], int lane, F tol, int& my_id) {
  const F none = -(F)INFINITY;
  bool sure = true;
  F last = none;
  my_id = -1;
  for (int j = 0; j <= a.k; ++j) {
    F b = none;
    int idx = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] > b) {
        b = key[i];
        idx = lane + 32 * i;
      }
    warp_best(b, idx);
    if (b == none) break;
    if (j && !(last - b > tol)) sure = false;
    if (j == a.k) break;
    if (lane == j) my_id = idx;
    if ((idx & 31) == lane) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == (idx >> 5)) key[i] = none;
    }
    last = b;
    if (j == a.k - 1 && tol < (F)0) break;  // exact keys: nothing is compared with the next one
  }
  return sure;
}

// log sigmoid(l), without overflow
__device__ __forceinline__ float log_sigmoid(float l) { return fminf(l, 0.0f) - log1pf(expf(-fabsf(l))); }
__device__ __forceinline__ float sigmoid_f(float l) { return 1.0f / (1.0f + expf(-l)); }

// A NaN logit switches its expert off, as -inf does.
template <typename L>
__device__ __forceinline__ float one_logit(const RouteArgs& a, int64_t t, int e) {
  const float v = load_logit(reinterpret_cast<const L*>(a.logits) + t * a.E + e);
  return v == v ? v : -INFINITY;
}
template <typename L, int V>
__device__ __forceinline__ void load_row(const RouteArgs& a, int64_t t, int lane, float (&l)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < a.E ? one_logit<L>(a, t, e) : -INFINITY;
  }
}

// The whole selection of a token again, in 64 bits where keys are scores, else of the 32-bit
// logits in full.  It reads the row itself and is kept out of line, so that its registers do
// not count against the usual path.
template <typename L, int V, int SCORE>
__device__ __noinline__ int select_again(const RouteArgs& a, int64_t t, int lane) {
  float l[V];
  load_row<L, V>(a, t, lane, l);
  int id;
  if (!a.bias && !(a.groups > 1 && a.group_top == 2)) {
    if (a.groups > 1) keep_groups<float, V>(a, l, lane, -1.0f);
    pick<float, V>(a, l, lane, -1.0f, id);
    return id;
  }
  float m = 0.0f;
  double sum = 1.0;
  if (SCORE == 0) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (l[i] > -INFINITY) sum += exp(below((double)l[i], (double)m));
    sum = warp_sum(sum);
  }
  double key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = -INFINITY;
    if (l[i] > -INFINITY) {
      double k = SCORE == 0 ? exp(below((double)l[i], (double)m)) / sum : 1.0 / (1.0 + exp(-(double)l[i]));
      if (a.bias) k += (double)a.bias[lane + 32 * i];
      if (k == k) key[i] = k;
    }
  }
  if (a.groups > 1) keep_groups<double, V>(a, key, lane, -1.0);
  pick<double, V>(a, key, lane, -1.0, id);
  return id;
}

// The sum, or the maximum, over aligned groups of n neighbouring lanes, n a power of two.
__device__ __forceinline__ float lanes_max(float v, int n) {
  for (int o = n >> 1; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float lanes_sum(float v, int n) {
  for (int o = n >> 1; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// The j-th lane of n (a power of two, at least k) that share token t holds its j-th chosen
// expert (-1: none): its weight, and both stored.  t < 0: no token.  m and inv: the row's
// largest logit and the inverse of its sum of exponentials (softmax weights that are not
// renormalised).
template <typename L, int SCORE>
__device__ __forceinline__ void store_choice(const RouteArgs& a, int64_t t, int lane, int n, int id, float m,
                                             float inv) {
  const int j = lane & (n - 1);
  const bool mine_to_store = t >= 0 && j < a.k, on = mine_to_store && id >= 0;
  const float mine = on ? one_logit<L>(a, t, id) : -INFINITY;  // read again, from L1
  float w;
  if (a.renorm) {
    // s_j / sum s_i: softmax's as exponentials relative to the largest chosen logit; sigmoids
    // as they are, unless one is so small (below e^-60) that only its logarithm is safe
    const unsigned small = SCORE == 0 ? 0u : __ballot_sync(kFull, on && mine < -60.0f);
    float ex = SCORE == 0 ? 0.0f : on ? sigmoid_f(mine) : 0.0f;
    if (SCORE == 0 || small) {
      const float ls = on ? (SCORE == 0 ? mine : log_sigmoid(mine)) : -INFINITY;
      const float mx = lanes_max(ls, n);
      if (SCORE == 0 || (small >> (lane - j) & (0xffffffffu >> (32 - n)))) ex = on ? expf(below(ls, mx)) : 0.0f;
    }
    w = ex / lanes_sum(ex, n);
  } else {
    w = SCORE == 0 ? expf(below(mine, m)) * inv : sigmoid_f(mine);
  }
  if (mine_to_store) {
    a.ids[t * a.k + j] = id;
    a.weights[t * a.k + j] = on ? a.scale * w : 0.0f;
  }
}

// ------------------------------------------------------------------ V neighbours a lane

__device__ __forceinline__ void order_two(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}
// Largest first.
__device__ __forceinline__ void sort_lane(uint32_t (&)[1]) {}
__device__ __forceinline__ void sort_lane(uint32_t (&v)[2]) { order_two(v[0], v[1]); }
__device__ __forceinline__ void sort_lane(uint32_t (&v)[4]) {
  order_two(v[0], v[1]);
  order_two(v[2], v[3]);
  order_two(v[0], v[2]);
  order_two(v[1], v[3]);
  order_two(v[1], v[2]);
}
__device__ __forceinline__ void sort_lane(uint32_t (&v)[8]) {  // odd-even merge of two sorted fours
#pragma unroll
  for (int h = 0; h < 8; h += 4) {
    order_two(v[h], v[h + 1]);
    order_two(v[h + 2], v[h + 3]);
    order_two(v[h], v[h + 2]);
    order_two(v[h + 1], v[h + 3]);
    order_two(v[h + 1], v[h + 2]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) order_two(v[i], v[i + 4]);
  order_two(v[2], v[4]);
  order_two(v[3], v[5]);
  order_two(v[1], v[2]);
  order_two(v[3], v[4]);
  order_two(v[5], v[6]);
}

__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

template <int V>
__device__ __forceinline__ void load_lane(const float* row, int e0, int E, bool vec, float (&l)[V]) {
  if (vec && e0 + V <= E) {
    if constexpr (V == 8 || V == 4) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(row + e0 + i);
        l[i] = v.x;
        l[i + 1] = v.y;
        l[i + 2] = v.z;
        l[i + 3] = v.w;
      }
      return;
    } else if constexpr (V == 2) {
      const float2 v = *reinterpret_cast<const float2*>(row + e0);
      l[0] = v.x;
      l[1] = v.y;
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = e0 + i < E ? row[e0 + i] : -INFINITY;
}
template <int V>
__device__ __forceinline__ void load_lane(const __nv_bfloat16* row, int e0, int E, bool vec, float (&l)[V]) {
  if constexpr (V > 1) {
    if (vec && e0 + V <= E) {
      uint32_t w[V / 2];
      if constexpr (V == 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + e0);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      } else if constexpr (V == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(row + e0);
        w[0] = v.x, w[1] = v.y;
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(row + e0);
      }
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        l[2 * i] = __uint_as_float(w[i] << 16);
        l[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = e0 + i < E ? __bfloat162float(row[e0 + i]) : -INFINITY;
}

// Bits of a double that compare as integers as the doubles do.
__device__ __forceinline__ int64_t ordered_64(double d) {
  const int64_t u = __double_as_longlong(d + 0.0);
  return u ^ ((u >> 63) & 0x7fffffffffffffffll);
}

// Keys in 64 bits (logits: in full), one to a lane, of the experts whose approximate key is at
// least this lane's `floor`: the c-th such expert e goes to lane c.  Returns how many there
// are; more than 32 do not fit.
template <typename L, int V, int SCORE, bool scored>
__device__ __forceinline__ int candidates(const RouteArgs& a, int64_t t, int lane, float floor, int& e, double& key) {
  float l[V];
  load_lane<V>(reinterpret_cast<const L*>(a.logits) + t * a.E, lane * V, a.E, false, l);
  float m = 0.0f;
  double sum = 1.0;
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = l[i] == l[i] ? l[i] : -INFINITY;
  if (scored && SCORE == 0) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += l[i] > -INFINITY ? exp(below((double)l[i], (double)m)) : 0.0;
    sum = warp_sum(sum);
  }
  int total = 0, src = -1, part = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float k = l[i];
    if (scored && l[i] > -INFINITY) {
      k = SCORE == 0 ? __expf(below(l[i], m)) / (float)sum : sigmoid_f(l[i]);
      if (a.bias) k += a.bias[lane * V + i];
    }
    for (unsigned mask = __ballot_sync(kFull, k > -INFINITY && k >= floor); mask; mask &= mask - 1, ++total)
      if (lane == total) {
        src = __ffs(mask) - 1;
        part = i;
      }
  }
  float mine = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float x = __shfl_sync(kFull, l[i], src < 0 ? 0 : src);
    if (part == i) mine = x;
  }
  e = src < 0 ? 0x7fffffff : src * V + part;
  key = -INFINITY;
  if (src >= 0) {
    key = mine;
    if (scored) {
      key = SCORE == 0 ? exp(below((double)mine, (double)m)) / sum : 1.0 / (1.0 + exp(-(double)mine));
      if (a.bias) key += (double)a.bias[e];
    }
  }
  return total;
}

// The kept groups, a bit each, where 32-bit ranks could not decide: ranks again from every
// group's candidates.  0 if they do not fit.
template <typename L, int V, int SCORE, bool scored>
__device__ __noinline__ unsigned groups_again(const RouteArgs& a, int64_t t, int lane, float floor) {
  int e;
  double key;
  const int total = candidates<L, V, SCORE, scored>(a, t, lane, floor, e, key);
  if (total > 32) return 0;
  const int64_t none = ordered_64(-INFINITY);
  const int64_t o = ordered_64(key);
  int64_t b1 = none, b2 = none;
  double d1 = -INFINITY, d2 = -INFINITY;
  for (int c = 0; c < total; ++c) {
    const int64_t k = __shfl_sync(kFull, o, c);
    const double d = __shfl_sync(kFull, key, c);
    if (__shfl_sync(kFull, e, c) / a.group_size != lane) continue;
    if (k > b1) {
      b2 = b1, d2 = d1;
      b1 = k, d1 = d;
    } else if (k > b2) {
      b2 = k, d2 = d;
    }
  }
  const int64_t rank = ordered_64(a.group_top == 2 && a.group_size > 1 ? rank_of_two(d1, d2) : d1);
  int better = 0;
  for (int g = 0; g < a.groups; ++g) {
    const int64_t r = __shfl_sync(kFull, rank, g);
    better += r > rank || (r == rank && g < lane);
  }
  return __ballot_sync(kFull, lane < a.groups && better < a.group_limit);
}

// The chosen experts (lane j: the j-th), where 32-bit keys could not decide: the candidates
// from `least` on, the k-th key's approximation less its error, in the kept groups (this
// lane's among them or not).  -2 in every lane if they do not fit, or are not the n that there
// have to be.
template <typename L, int V, int SCORE, bool scored>
__device__ __noinline__ int order_again(const RouteArgs& a, int64_t t, int lane, bool keep, float least, int n) {
  int e;
  double key;
  const int total = candidates<L, V, SCORE, scored>(a, t, lane, keep ? least : NAN, e, key);
  if (total > 32 || total < n) return -2;
  const int64_t o = ordered_64(key);
  int better = 0;
  for (int c = 0; c < total; ++c) {
    const int64_t k = __shfl_sync(kFull, o, c);
    const int x = __shfl_sync(kFull, e, c);
    better += k > o || (k == o && x < e);
  }
  int id = -1;
  for (int c = 0; c < total; ++c) {
    const int place = __shfl_sync(kFull, better, c), x = __shfl_sync(kFull, e, c);
    if (place == lane) id = x;
  }
  return lane < a.k ? id : -1;
}

constexpr int kRouteBlocks = 4;  // resident blocks of route_kernel on an SM

// scored: keys are scores, or sums of two (a bias, or group_top = 2 with groups); else logits.
// `vec`: rows start at multiples of V elements.  A group is group_size / V neighbouring lanes,
// a power of two of them (one group: any size).
template <typename L, int V, int SCORE, bool scored, bool grouped>
__global__ void __launch_bounds__(256, kRouteBlocks) route_kernel(const __grid_constant__ RouteArgs a, int vec) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, e0 = lane * V;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  constexpr uint32_t kLow = V - 1;
  float bias[V], next[V];
  float bias_most = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bias[i] = a.bias && e0 + i < a.E ? a.bias[e0 + i] : 0.0f;
    if (fabsf(bias[i]) < INFINITY) bias_most = fmaxf(bias_most, fabsf(bias[i]));
  }
  // a group's lanes, this lane's group and the group's first lane
  const int lanes = a.group_size / V > 0 ? a.group_size / V : 1, mine = lane / lanes, leader = mine * lanes;
  bias_most = warp_max(bias_most);
  const int share = a.k > 1 ? 1 << (32 - __clz(a.k - 1)) : 1;  // lanes of a choice
  int held = 0, their_id = -1;
  int64_t their_t = -1;
  float their_m = 0.0f, their_inv = 0.0f;
  load_lane<V>(reinterpret_cast<const L*>(a.logits) + t * a.E, e0, a.E, vec, next);
  for (; t < a.T; t += warps) {
    float l[V];
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = SCORE == 0 && !(next[i] == next[i]) ? -INFINITY : next[i];
    if (t + warps < a.T) load_lane<V>(reinterpret_cast<const L*>(a.logits) + (t + warps) * a.E, e0, a.E, vec, next);
    // softmax's largest logit and sum, where a score of its own is needed
    float m = 0.0f, inv = 0.0f;
    if (SCORE == 0 && (scored || !a.renorm)) {
      m = l[0];
#pragma unroll
      for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
      m = warp_max(m);
      float sum = 0.0f;
      if (m > -INFINITY) {
        const bool finite = m < INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float ex = finite ? expf(l[i] - m) : l[i] == m ? 1.0f : 0.0f;
          sum += ex;
          if (scored && l[i] > -INFINITY) l[i] = ex;  // -inf stays -inf, off
        }
      }
      inv = 1.0f / warp_sum(sum);
    }
    // Keys.  A bound on how far the difference of two may be off (tol), besides the low bits:
    // sigmoid: the fast exponential (2 + 1.2 |l| ulp, times s (1 - s)) and division (2 ulp), the
    // addition: 3.7e-7 a key.  softmax: expf of l - m (2 ulp and the argument's rounding), at most 37
    // additions in the sum, a product: 3e-6 of a score of at most inv.  The bias adds half an ulp, the low
    // bits 7 ulp of the larger key.
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float k = l[i];
      if (scored) {
        k = SCORE == 0 ? l[i] * inv : __fdividef(1.0f, 1.0f + __expf(-l[i]));
        k += bias[i];
      }
      // -inf and NaN logits (or biases) are off
      key[i] = l[i] > -INFINITY && k > -INFINITY ? ((ordered(k) & ~kLow) | (kLow - i)) : 0u;
    }
    sort_lane(key);
    const float most = SCORE == 0 ? inv : 1.0f;  // a score is at most
    const float tol = scored ? (SCORE == 0 ? 6.5e-6f * inv : 8e-7f) + 1.1e-6f * (most + bias_most) : 0.0f;
    bool keep = true;   // this lane's group is among the kept ones
    bool lost = false;  // nothing here can decide: the whole selection again
    if (grouped) {
      uint32_t b1 = key[0], b2 = V > 1 ? key[V > 1 ? 1 : 0] : 0u;
      for (int o = 1; o < lanes; o <<= 1) {
        const uint32_t c1 = __shfl_xor_sync(kFull, b1, o), c2 = __shfl_xor_sync(kFull, b2, o);
        b2 = max(min(b1, c1), max(b2, c2));
        b1 = max(b1, c1);
      }
      auto value = [](uint32_t k) { return k ? unordered(k & ~kLow) : -INFINITY; };
      float rank = value(b1);
      if (a.group_top == 2 && a.group_size > 1) rank = rank_of_two(rank, value(b2));
      // the groups in order of rank, of equal ones the lower first; a group's lanes hold the same
      const bool real = mine < a.groups;
      uint32_t left = real ? ordered(rank) : 0u, best, last = 0u;
      keep = false;
      for (int n = 0;; ++n) {
        best = __reduce_max_sync(kFull, left);
        if (best == 0u || n == a.group_limit) break;
        last = best;
        const int who = __ffs(__ballot_sync(kFull, left == best)) - 1;
        if (leader == (who & -lanes)) {
          keep = true;
          left = 0u;
        }
      }
      // the closest pair across the border: scores, by the bound; 32-bit logits, by equality but
      // for the low bits
      const float low = unordered(last), high = best ? unordered(best) : -INFINITY;
      if ((scored || sizeof(L) == 4) && high > -INFINITY && !(scored ? low - high > 2.0f * tol : low != high)) {
        const float floor = value(a.group_top == 2 && a.group_size > 1 ? b2 : b1) - 4.0f * tol;
        const unsigned bits = groups_again<L, V, SCORE, scored>(a, t, lane, real ? floor : NAN);
        lost = bits == 0;
        keep = real && ((bits >> mine) & 1u);
      }
      if (!keep) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = 0u;
      }
    }
    // lane j: the j-th chosen key and its lane; `best`: the first one left out
    uint32_t got = 0u, best;
    int from = 0, n = 0;
    for (;; ++n) {
      const uint32_t head = key[0] | kLow;
      best = __reduce_max_sync(kFull, head);
      if (best == kLow || n == a.k) break;  // none left, or enough
      const int who = __ffs(__ballot_sync(kFull, head == best)) - 1;  // equal keys: the lowest expert
      const uint32_t won = __shfl_sync(kFull, key[0], who);
      if (lane == n) {
        got = won;
        from = who;
      }
      if (lane == who) {
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
        key[V - 1] = 0u;
      }
    }
    int id = lane < n ? from * V + (int)(~got & kLow) : -1;
    if (scored || sizeof(L) == 4) {
      // a chosen key against the one after it; one of +inf (a bias) is never far enough from it
      const uint32_t below = __shfl_down_sync(kFull, got, 1) | kLow, after = lane == n - 1 ? best : below;
      const bool close = scored ? !(unordered(got | kLow) - unordered(after) > tol) : (got | kLow) == after;
      if (__any_sync(kFull, lane < n && after != kLow && close) && !lost) {
        const uint32_t last = __shfl_sync(kFull, got, n - 1);
        const float least = unordered(scored ? min(last | kLow, ordered(INFINITY)) : last & ~kLow);
        id = order_again<L, V, SCORE, scored>(a, t, lane, keep, least - 4.0f * tol, n);
        lost = id == -2;
      }
    }
    if (__any_sync(kFull, lost)) id = select_again<L, V, SCORE>(a, t, lane);
    // the choices of 32 / share tokens are stored together
    const int moved = __shfl_sync(kFull, id, lane & (share - 1));
    if ((lane & -share) == held) {
      their_t = t;
      their_id = moved;
      their_m = m;
      their_inv = inv;
    }
    held += share;
    if (held == 32 || t + warps >= a.T) {
      store_choice<L, SCORE>(a, their_t, lane, share, their_id, their_m, their_inv);
      held = 0;
      their_t = -1;
    }
  }
}

// ------------------------------------------------------------------ any count and grouping

template <typename L, int V, int SCORE>
__global__ void __launch_bounds__(256) route_any_kernel(const __grid_constant__ RouteArgs a) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  float l[V], key[V];
  load_row<L, V>(a, t, lane, l);
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
  m = warp_max(m);
  // 32-bit scores are needed for keys with a bias, for ranks that add two scores, and for
  // softmax weights that are not renormalised
  const bool scored = a.bias != nullptr || (a.groups > 1 && a.group_top == 2);
  float sum = 0.0f;
  if (SCORE == 0 && (scored || !a.renorm)) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = expf(below(l[i], m));
      if (lane + 32 * i < a.E) sum += key[i];
    }
    sum = warp_sum(sum);
  }
  // A bound on how far two 32-bit keys' difference may be off.  sigmoid: expf (2 ulp), an
  // addition and a division each half an ulp, of a value of at most 1: 3.6e-7 a key.
  // softmax: the same, the argument's rounding, and the sum's (at most 37 additions,
  // 2.3e-6), of a value of at most 1/sum.  The bias adds half an ulp of the key; a rank
  // adds two keys.
  float tol = -1.0f;
  if (scored) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 32 * i;
      key[i] = SCORE == 0 ? key[i] / sum : sigmoid_f(l[i]);
      if (a.bias && e < a.E) key[i] += a.bias[e];
      if (l[i] == -INFINITY || key[i] != key[i]) key[i] = -INFINITY;
      if (key[i] > -INFINITY) top = fmaxf(top, fabsf(key[i]));
    }
    top = warp_max(top);
    tol = (SCORE == 0 ? 6e-6f / sum : 1e-6f) + 2.4e-7f * top;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = l[i] == l[i] ? l[i] : -INFINITY;
  }
  bool sure = true;
  if (a.groups > 1) sure = keep_groups<float, V>(a, key, lane, scored ? 2.0f * tol : -1.0f);
  int id;
  sure = pick<float, V>(a, key, lane, tol, id) && sure;
  if (scored && !sure) id = select_again<L, V, SCORE>(a, t, lane);
  store_choice<L, SCORE>(a, t, lane, 32, id, m, 1.0f / sum);
}

// ------------------------------------------------------------------ gradient

// With q_j = s_j / sum of chosen s (renorm) the chosen experts' gradients need nothing of
// the others, for softmax too (its denominator cancels):
//   softmax  dl_j = scale q_j (dw_j - sum_i q_i dw_i)
//   sigmoid  the same, times 1 - s_j
// Without: softmax dl_e = p_e (scale dw_e [e chosen] - scale sum_j p_j dw_j), sigmoid
// dl_j = scale dw_j s_j (1 - s_j).  All other gradients are zero, so that only softmax
// without renorm has to read the row.
//
// Lane j of a token's N lanes holds the j-th chosen expert.  The chosen's part of its gradient,
// and softmax's common term scale sum_j p_j dw_j in every lane.
template <int SCORE, int N = 32>
__device__ __forceinline__ float chosen_grad(const RouteArgs& a, bool on, float mine, float dw, float m, float inv,
                                             float& inner) {
  inner = 0.0f;
  float g = 0.0f;
  if (a.renorm) {
    const float ls = on ? (SCORE == 0 ? mine : log_sigmoid(mine)) : -INFINITY;
    const float mx = warp_max<N>(ls);
    const float ex = on ? expf(below(ls, mx)) : 0.0f;
    const float q = ex / warp_sum<N>(ex);
    const float mean = warp_sum<N>(on ? q * dw : 0.0f);
    if (on) g = a.scale * q * (dw - mean);
    if (SCORE == 1 && on) g *= sigmoid_f(-mine);
  } else if (SCORE == 0) {
    const float p = on ? expf(below(mine, m)) * inv : 0.0f;
    inner = a.scale * warp_sum<N>(on ? p * dw : 0.0f);
    if (on) g = a.scale * dw * p;
  } else if (on) {
    g = a.scale * dw * sigmoid_f(mine) * sigmoid_f(-mine);
  }
  return g;
}

// Lane j's chosen expert (-1: none, or switched off), its logit and the gradient of its weight.
template <typename L>
__device__ __forceinline__ bool load_chosen(const RouteArgs& a, int64_t t, int lane, int& id, float& mine, float& dw) {
  id = -1;
  dw = 0.0f;
  if (lane < a.k) {
    id = a.ids[t * a.k + lane];
    if (id < 0 || id >= a.E) id = -1;
    dw = a.weights[t * a.k + lane];
  }
  mine = id >= 0 ? one_logit<L>(a, t, id) : -INFINITY;
  return mine > -INFINITY;
}

// An expert that a token was given twice gets the sum of both, from the first of the two
// lanes, which is the one that stores (returned).  key: equal for equal experts of a token.
template <int N>
__device__ __forceinline__ bool first_of_equals(int lane, int key, float& g) {
  const unsigned same = __match_any_sync(kFull, key);
  if (__any_sync(kFull, __popc(same) > 1)) {
    float total = 0.0f;
    for (int j = 0; j < N; ++j) {
      const int from = (lane & ~(N - 1)) + j;
      const float v = __shfl_sync(kFull, g, from);
      if ((same >> from) & 1u) total += v;
    }
    g = total;
  }
  return (same & ((1u << lane) - 1)) == 0;
}

// Gradients that are zero but for the chosen experts', rows of whole 16-byte pieces: a token
// takes N >= k lanes, a warp 32 / N tokens; rows are zeroed, then the chosen's values stored
// over them.  32768 tokens x 256 experts, 8 a token: 10 us, 20 us for route_grad_kernel.
template <typename L, int SCORE, int N>
__global__ void __launch_bounds__(256) route_grad_chosen_kernel(const __grid_constant__ RouteArgs a) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, group = lane / N;
  const int64_t t0 = ((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * (32 / N), t = t0 + group;
  if (t0 >= a.T) return;
  int id = -1;
  float mine = -INFINITY, dw = 0.0f;
  if (t < a.T) load_chosen<L>(a, t, lane & (N - 1), id, mine, dw);
  const bool on = mine > -INFINITY;
  const int64_t rows = min((int64_t)(32 / N), a.T - t0);
  uint4* out = reinterpret_cast<uint4*>(reinterpret_cast<L*>(a.dlogits) + t0 * a.E);
  const int pieces = (int)(rows * a.E * (int64_t)sizeof(L) / 16);
#pragma unroll 4
  for (int c = lane; c < pieces; c += 32) out[c] = make_uint4(0u, 0u, 0u, 0u);
  float inner;
  float g = chosen_grad<SCORE, N>(a, on, mine, dw, 0.0f, 0.0f, inner);
  const bool first = first_of_equals<N>(lane, on ? id * 32 + group : -1 - lane, g);
  __syncwarp();  // the rows are written
  if (on && first) store_logit(reinterpret_cast<L*>(a.dlogits) + t * a.E + id, g);
}

// softmax without renorm: every expert's gradient, rows of whole 16-byte pieces, at most C of
// them a lane.
template <typename L, int C>
__global__ void __launch_bounds__(256) route_grad_rows_kernel(const __grid_constant__ RouteArgs a) {
  constexpr int W = 16 / sizeof(L);
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const L* row = reinterpret_cast<const L*>(a.logits) + t * a.E;
  float l[C * W];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float v[W];
    load_lane<W>(row, (c * 32 + lane) * W, a.E, true, v);
#pragma unroll
    for (int i = 0; i < W; ++i) l[c * W + i] = v[i] == v[i] ? v[i] : -INFINITY;
  }
  int id;
  float mine, dw;
  const bool on = load_chosen<L>(a, t, lane, id, mine, dw);
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < C * W; ++i) m = fmaxf(m, l[i]);
  m = warp_max(m);
  if (m == -INFINITY) m = 0.0f;  // every expert switched off: zeros
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < C * W; ++i) {
    l[i] = expf(below(l[i], m));
    sum += l[i];
  }
  sum = warp_sum(sum);
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  float inner;
  float g = chosen_grad<0>(a, on, mine, dw, m, inv, inner);
  L* out = reinterpret_cast<L*>(a.dlogits) + t * a.E;
  const float common = -inner * inv;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e0 = (c * 32 + lane) * W;
    uint32_t p[4];
    if constexpr (W == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = __float_as_uint(common * l[c * W + i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(common * l[c * W + 2 * i], common * l[c * W + 2 * i + 1]);
        p[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    if (e0 < a.E) *reinterpret_cast<uint4*>(out + e0) = make_uint4(p[0], p[1], p[2], p[3]);
  }
  const bool first = first_of_equals<32>(lane, on ? id : -1 - lane, g);
  __syncwarp();  // the row is written
  if (on && first) store_logit(out + id, g + common * expf(below(mine, m)));
}

// Any count of experts.
template <typename L, int V, int SCORE>
__global__ void __launch_bounds__(256) route_grad_kernel(const __grid_constant__ RouteArgs a) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  float l[V];
  load_row<L, V>(a, t, lane, l);
  int id;
  float mine, dw;
  const bool on = load_chosen<L>(a, t, lane, id, mine, dw);
  float m = 0.0f, inv = 0.0f;
  if (SCORE == 0 && !a.renorm) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 32 * i < a.E) sum += expf(below(l[i], m));
    inv = 1.0f / warp_sum(sum);
  }
  float inner;
  const float g = chosen_grad<SCORE>(a, on, mine, dw, m, inv, inner);
  float d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    d[i] = 0.0f;
    if (SCORE == 0 && !a.renorm && l[i] != -INFINITY) d[i] = -inner * expf(below(l[i], m)) * inv;
  }
  for (int j = 0; j < a.k; ++j) {
    const int e = __shfl_sync(kFull, on ? id : -1, j);
    const float v = __shfl_sync(kFull, g, j);
    if (e >= 0 && (e & 31) == lane) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == (e >> 5)) d[i] += v;
    }
  }
  L* row = reinterpret_cast<L*>(a.dlogits) + t * a.E;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    if (e < a.E) store_logit(row + e, d[i]);
  }
}

// ------------------------------------------------------------------ launches

template <typename L, int V, int SCORE>
cudaError_t launch_lanes(bool scored, bool grouped, dim3 g, cudaStream_t s, const RouteArgs& a, int vec) {
  if (scored)
    return grouped ? launch(route_kernel<L, V, SCORE, true, true>, g, 256, 0, s, a, vec)
                   : launch(route_kernel<L, V, SCORE, true, false>, g, 256, 0, s, a, vec);
  return grouped ? launch(route_kernel<L, V, SCORE, false, true>, g, 256, 0, s, a, vec)
                 : launch(route_kernel<L, V, SCORE, false, false>, g, 256, 0, s, a, vec);
}

template <typename L, int SCORE>
cudaError_t launch_grad_rows(const RouteArgs& a, dim3 rows, cudaStream_t s) {
  if (SCORE == 0 && !a.renorm) {
    const int c = (a.E * (int)sizeof(L) + 511) / 512;
    if (c <= 1) return launch(route_grad_rows_kernel<L, 1>, rows, 256, 0, s, a);
    if (c <= 2) return launch(route_grad_rows_kernel<L, 2>, rows, 256, 0, s, a);
    if (c <= 4) return launch(route_grad_rows_kernel<L, 4>, rows, 256, 0, s, a);
    return launch(route_grad_rows_kernel<L, 8>, rows, 256, 0, s, a);
  }
  const int n = a.k <= 4 ? 4 : a.k <= 8 ? 8 : a.k <= 16 ? 16 : 32;
  const dim3 g((unsigned)((a.T * n + 255) / 256));
  if (n == 4) return launch(route_grad_chosen_kernel<L, SCORE, 4>, g, 256, 0, s, a);
  if (n == 8) return launch(route_grad_chosen_kernel<L, SCORE, 8>, g, 256, 0, s, a);
  if (n == 16) return launch(route_grad_chosen_kernel<L, SCORE, 16>, g, 256, 0, s, a);
  return launch(route_grad_chosen_kernel<L, SCORE, 32>, g, 256, 0, s, a);
}

template <typename L, int SCORE, bool GRAD>
cudaError_t launch_route(const RouteArgs& a, int sms, cudaStream_t s) {
  const dim3 grid((unsigned)((a.T + 7) / 8));
  const int v = (a.E + 31) / 32;
  if (GRAD && a.E * sizeof(L) % 16 == 0) return launch_grad_rows<L, SCORE>(a, grid, s);
  // Up to 256 experts in groups of whole lanes, a power of two of them: neighbours in a lane;
  // warps go on to further tokens, so that the biases are read once.
  if (!GRAD && v <= 8) {
    const int V = v <= 1 ? 1 : v <= 2 ? 2 : v <= 4 ? 4 : 8, lanes = a.group_size / V;
    if (a.groups == 1 || (a.group_size % V == 0 && (lanes & (lanes - 1)) == 0)) {
      const dim3 g((unsigned)std::min<int64_t>(((a.T + 7) / 8), (int64_t)sms * kRouteBlocks));
      const int vec = a.E % V == 0;
      const bool grouped = a.groups > 1, scored = a.bias || (grouped && a.group_top == 2);
      if (V == 1) return launch_lanes<L, 1, SCORE>(scored, grouped, g, s, a, vec);
      if (V == 2) return launch_lanes<L, 2, SCORE>(scored, grouped, g, s, a, vec);
      if (V == 4) return launch_lanes<L, 4, SCORE>(scored, grouped, g, s, a, vec);
      return launch_lanes<L, 8, SCORE>(scored, grouped, g, s, a, vec);
    }
  }
#define CUSYNC_ROUTE(V)                                                                     \
  if (v <= V)                                                                               \
    return GRAD ? launch(route_grad_kernel<L, V, SCORE>, grid, 256, 0, s, a)                \
                : launch(route_any_kernel<L, V, SCORE>, grid, 256, 0, s, a);
  CUSYNC_ROUTE(1)
  CUSYNC_ROUTE(2)
  CUSYNC_ROUTE(4)
  CUSYNC_ROUTE(8)
  CUSYNC_ROUTE(16)
  CUSYNC_ROUTE(32)
#undef CUSYNC_ROUTE
  return cudaErrorInvalidValue;
}

template <typename L>
cudaError_t route_logits(const RouteArgs& a, bool softmax, bool grad, int sms, cudaStream_t s) {
  if (grad) return softmax ? launch_route<L, 0, true>(a, sms, s) : launch_route<L, 1, true>(a, sms, s);
  return softmax ? launch_route<L, 0, false>(a, sms, s) : launch_route<L, 1, false>(a, sms, s);
}

}  // namespace moe
}  // namespace cusync
