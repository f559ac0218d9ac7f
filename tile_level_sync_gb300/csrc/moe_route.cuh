// The router of a mixture-of-experts layer and its gradient: one warp per token.
//
// A lane holds experts lane, lane + 32, ... (V of them) in registers, so a row of logits is
// read once, coalesced, at any expert count.  Scores are s = softmax(l) or sigmoid(l); the
// choice goes by key = s + bias.  The largest key is found by one pass over a lane's
// registers and two warp reductions (of the key's ordered bits, then of the index among
// equal keys), so equal keys go to the lowest index.
//
// Without a bias the keys are the logits themselves (both scores grow with the logit): the
// comparison is exact.  With one, 32-bit keys carry the rounding of the exponential, the
// sum and the addition; where two neighbours in the chosen order (or the last chosen and
// the first left out, or two groups' ranks) are closer than a bound on that error, the
// token's selection is done again with 64-bit scores.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ptx.cuh"

namespace cusync {
namespace moe {

constexpr unsigned kFull = 0xffffffffu;

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;        // route: out; gradient: dweights (in)
  void* dlogits;
  int64_t T;
  int32_t E, k, groups, group_size, group_limit, group_top;
  int32_t renorm;
  float scale;
};

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Bits that compare as unsigned integers as the floats do; both zeros alike.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
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
      r = m1 + b2;
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

template <int V, int SCORE>
__device__ __forceinline__ void keys_64(const RouteArgs& a, const float (&l)[V], int lane, float m, double (&key)[V]) {
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = SCORE == 0 ? exp((double)l[i] - (double)m) : 1.0 / (1.0 + exp(-(double)l[i]));
    sum += key[i];
  }
  if (SCORE == 0) sum = warp_sum(sum);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    if (SCORE == 0) key[i] /= sum;
    if (a.bias && e < a.E) key[i] += (double)a.bias[e];
    if (l[i] == -INFINITY || key[i] != key[i]) key[i] = -INFINITY;
  }
}

// The selection again, in 64 bits; kept out of line so that its registers do not count
// against the usual path.
template <int V, int SCORE>
__device__ __noinline__ int pick_64(const RouteArgs& a, const float (&l)[V], int lane, float m) {
  double key[V];
  keys_64<V, SCORE>(a, l, lane, m, key);
  if (a.groups > 1) keep_groups<double, V>(a, key, lane, -1.0);
  int id;
  pick<double, V>(a, key, lane, -1.0, id);
  return id;
}

template <typename L, int V, int SCORE>
__global__ void __launch_bounds__(256) route_kernel(RouteArgs a) {
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
      key[i] = expf(l[i] - m);
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
  if (scored && !sure) id = pick_64<V, SCORE>(a, l, lane, m);
  // weights: lane j holds the j-th chosen expert (its logit read again, from L1)
  const bool on = lane < a.k && id >= 0;
  const float mine = on ? one_logit<L>(a, t, id) : -INFINITY;
  float w;
  if (a.renorm) {
    // s_j / sum s_i = exp(log s_j) / sum exp(log s_i), taken relative to the largest chosen
    // score: no underflow, whatever the others are
    const float ls = on ? (SCORE == 0 ? mine : log_sigmoid(mine)) : -INFINITY;
    const float mx = warp_max(ls);
    const float ex = on ? expf(ls - mx) : 0.0f;
    w = ex / warp_sum(ex);
  } else {
    w = SCORE == 0 ? expf(mine - m) / sum : sigmoid_f(mine);
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = id;
    a.weights[t * a.k + lane] = on ? a.scale * w : 0.0f;
  }
}

// With q_j = s_j / sum of chosen s (renorm) the chosen experts' gradients need nothing of
// the others, for softmax too (its denominator cancels):
//   softmax  dl_j = scale q_j (dw_j - sum_i q_i dw_i)
//   sigmoid  the same, times 1 - s_j
// Without: softmax dl_e = p_e (scale dw_e [e chosen] - scale sum_j p_j dw_j), sigmoid
// dl_j = scale dw_j s_j (1 - s_j).  All other gradients are zero.
template <typename L, int V, int SCORE>
__global__ void __launch_bounds__(256) route_grad_kernel(RouteArgs a) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  float l[V];
  load_row<L, V>(a, t, lane, l);
  int id = -1;
  float dw = 0.0f;
  if (lane < a.k) {
    id = a.ids[t * a.k + lane];
    if (id < 0 || id >= a.E) id = -1;
    dw = a.weights[t * a.k + lane];
  }
  const float mine = id >= 0 ? one_logit<L>(a, t, id) : -INFINITY;
  const bool on = mine > -INFINITY;
  float m = 0.0f, inv = 0.0f;
  if (SCORE == 0 && !a.renorm) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 32 * i < a.E) sum += expf(l[i] - m);
    inv = 1.0f / warp_sum(sum);
  }
  float g = 0.0f, inner = 0.0f;  // this lane's chosen expert's gradient; softmax's common term
  if (a.renorm) {
    const float ls = on ? (SCORE == 0 ? mine : log_sigmoid(mine)) : -INFINITY;
    const float mx = warp_max(ls);
    const float ex = on ? expf(ls - mx) : 0.0f;
    const float q = ex / warp_sum(ex);
    const float mean = warp_sum(on ? q * dw : 0.0f);
    if (on) g = a.scale * q * (dw - mean);
    if (SCORE == 1 && on) g *= sigmoid_f(-mine);
  } else if (SCORE == 0) {
    const float p = on ? expf(mine - m) * inv : 0.0f;
    inner = a.scale * warp_sum(on ? p * dw : 0.0f);
    if (on) g = a.scale * dw * p;
  } else if (on) {
    g = a.scale * dw * sigmoid_f(mine) * sigmoid_f(-mine);
  }
  float d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    d[i] = 0.0f;
    if (SCORE == 0 && !a.renorm && l[i] != -INFINITY) d[i] = -inner * expf(l[i] - m) * inv;
  }
  for (int j = 0; j < a.k; ++j) {
    const int e = __shfl_sync(kFull, id, j);
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

}  // namespace moe
}  // namespace cusync
