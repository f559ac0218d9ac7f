// The parts of an expert layer outside the tiled products: the sums over a token's
// experts, and the MLP of a few tokens without tiles.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "moe_gemm.cuh"
#include "moe_ptx.cuh"

namespace cusync {
namespace moe {

struct CombineArgs {
  int32_t* plan;
  const __half* rows;    // [slots, D], scaled by slot and 32 columns
  const uint8_t* scale;  // exponents of those powers of two (scale_at)
  const float* weights;  // [T, k], or null: plain sums
  void* out;             // [T, D] bf16
  const float* part;     // gradient: sums of dH h, [slots][parts]; null otherwise
  float* dweights;       // [T, k]
  int64_t slot_of;
  int32_t T, k, D, slots, parts, used;  // used: sums of a slot, of parts
};

struct DispatchArgs {
  int32_t* plan;
  const uint4 *x, *y;    // [T, chunks] of 16 bytes
  uint4 *xs, *ys;        // [slots, chunks]; y and ys may be null
  int64_t T, slot_of, counts, offsets;  // tokens; plan words
  int32_t k, E, chunks;
};

constexpr int kDispatchThreads = 256;

// Rows of X (and dY) into slot order: a thread reads 16 bytes of a token once and writes them
// to each of its slots.  Behind the tokens come the experts: zeros from an expert's last row up
// to the next multiple of kRowStep (the weight gradients sum over them).  4096 tokens of
// D = 2048 in 8 slots each: 22 us, 46 us for two tensors, at the rate of the writes; a warp
// per slot, which reads a token once for each slot, takes 32 and 62 us.
__global__ void __launch_bounds__(kDispatchThreads) dispatch_kernel(DispatchArgs a) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int64_t i = (int64_t)blockIdx.x * kDispatchThreads + threadIdx.x;
  const int64_t t = i / a.chunks, c = i - t * a.chunks;
  if (t < a.T) {
    const uint4 x = a.x[i], y = a.y ? a.y[i] : x;
    const int32_t* slots = a.plan + a.slot_of + t * a.k;
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
      const int32_t slot = slots[j];
      if (slot < 0) continue;
      const int64_t to = (int64_t)slot * a.chunks + c;
      a.xs[to] = x;
      if (a.y) a.ys[to] = y;
    }
  } else if (t < a.T + a.E) {
    const int e = (int)(t - a.T);
    const int32_t count = a.plan[a.counts + e];
    for (int32_t n = count; n % kRowStep; ++n) {
      const int64_t to = (a.plan[a.offsets + e] + (int64_t)n) * a.chunks + c;
      a.xs[to] = make_uint4(0, 0, 0, 0);
      if (a.y) a.ys[to] = make_uint4(0, 0, 0, 0);
    }
  }
}

constexpr int kCombineThreads = 256;

// out[t] = sum_j weights[t,j] rows[slot_of[t,j]], in the order of j, in fp32; one rounding.
// A block takes one token's next 8 * kCombineThreads columns.  With `part`, the first block
// of a token also adds up dweights from the column tiles' partial sums, in order.
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(CombineArgs a) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int64_t t = blockIdx.x;
  const int32_t* slots = a.plan + a.slot_of + t * a.k;
  const int c = (blockIdx.y * kCombineThreads + threadIdx.x) * 8;
  if (c < a.D) {
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.0f;
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
      const int32_t slot = slots[j];
      if (slot < 0) continue;
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(a.rows + (int64_t)slot * a.D + c));
      const float unit = __uint_as_float((uint32_t)a.scale[scale_at(a.slots, slot, c / 32)] << 23);
      const float w = a.weights ? a.weights[t * a.k + j] : 1.0f;
      const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&words[i]));
        s[2 * i] += w * (f.x * unit);
        s[2 * i + 1] += w * (f.y * unit);
      }
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + t * a.D + c) =
        make_uint4(pack2(s[0], s[1]), pack2(s[2], s[3]), pack2(s[4], s[5]), pack2(s[6], s[7]));
  }
  if (a.part && blockIdx.y == 0 && threadIdx.x < a.k) {
    const int32_t slot = slots[threadIdx.x];
    float s = 0.0f;
    if (slot >= 0)
      for (int i = 0; i < a.used; ++i) s += a.part[(int64_t)slot * a.parts + i];
    a.dweights[t * a.k + threadIdx.x] = s;
  }
}

struct SmallArgs {
  const uint16_t *X, *W1t, *W2t;
  const int32_t* ids;
  const float* weights;
  float* h;              // [A, N1] fp32
  uint16_t* Y;
  int32_t* err;          // the work buffer's error word
  int32_t T, k, E, D, N1;
};

__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ float dot8(const uint4& w, const uint4& x, float s) {
  s += lo16(w.x) * lo16(x.x);
  s += hi16(w.x) * hi16(x.x);
  s += lo16(w.y) * lo16(x.y);
  s += hi16(w.y) * hi16(x.y);
  s += lo16(w.z) * lo16(x.z);
  s += hi16(w.z) * hi16(x.z);
  s += lo16(w.w) * lo16(x.w);
  s += hi16(w.w) * hi16(x.w);
  return s;
}
__device__ __forceinline__ float dot8f(const uint4& w, const float4& x, const float4& y, float s) {
  s += lo16(w.x) * x.x;
  s += hi16(w.x) * x.y;
  s += lo16(w.y) * x.z;
  s += hi16(w.y) * x.w;
  s += lo16(w.z) * y.x;
  s += hi16(w.z) * y.y;
  s += lo16(w.w) * y.z;
  s += hi16(w.w) * y.w;
  return s;
}
__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }

constexpr int kSmallThreads = 256;
constexpr int kSmallBlocks = 4;  // of each kernel on an SM: both fit at once

// h[a][n] = act(X[t] . W1 rows of the chosen expert): a warp per (assignment, n) at a time.
// All blocks are resident from the start, so that those of small_down_kernel, which fit
// beside them, can begin to bring their weights to L2.
template <int ACT>
__global__ void __launch_bounds__(kSmallThreads, kSmallBlocks) small_up_kernel(SmallArgs a) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t units = (int64_t)a.T * a.k * a.N1, warps = (int64_t)gridDim.x * (kSmallThreads / 32);
  int64_t u = (int64_t)blockIdx.x * (kSmallThreads / 32) + (threadIdx.x >> 5);
  if (u == 0 && lane == 0) *a.err = 0;
  for (; u < units; u += warps) {
    const int as = (int)(u / a.N1), n = (int)(u - (int64_t)as * a.N1);
    const int e = a.ids[as];
    if ((unsigned)e >= (unsigned)a.E) continue;
    const uint16_t* x = a.X + (int64_t)(as / a.k) * a.D;
    const uint16_t* w = a.W1t + ((int64_t)e * (ACT == 1 ? 2 : 1) * a.N1 + n) * a.D;
    const uint16_t* v = w + (int64_t)a.N1 * a.D;
    float z = 0.0f, g = 0.0f;
#pragma unroll 8
    for (int c = lane * 8; c < a.D; c += 256) {
      const uint4 ww = ld_stream(w + c);
      uint4 vv;
      if (ACT == 1) vv = ld_stream(v + c);
      const uint4 xx = *reinterpret_cast<const uint4*>(x + c);
      z = dot8(ww, xx, z);
      if (ACT == 1) g = dot8(vv, xx, g);
    }
    z = warp_add(z);
    if (ACT == 1) g = warp_add(g);
    if (lane == 0) a.h[(int64_t)as * a.N1 + n] = ACT == 1 ? z * sigmoid_fast(z) * g : z * gelu_gate(z);
  }
}

// Y[t][d] = sum_j weights[t,j] W2[e_j][d] . h[t,j]: four warps per (t, d) at a time, each with
// a quarter of the token's experts, their sums added in the order of j.  It starts while
// small_up_kernel still runs (whose own start waited for the kernel before it, so the ids are
// there) and brings its first rows of W2t to L2 before it waits.
constexpr int kDownSplit = 4;
constexpr int kDownUnits = kSmallThreads / 32 / kDownSplit;  // (t, d) of a block at a time
__global__ void __launch_bounds__(kSmallThreads, kSmallBlocks) small_down_kernel(SmallArgs a) {
  __shared__ float sums[2][kDownUnits][kDownSplit];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = warp % kDownSplit, mine = warp / kDownSplit;
  const int j0 = part * a.k / kDownSplit, j1 = (part + 1) * a.k / kDownSplit;
  const int64_t units = (int64_t)a.T * a.D;
  int64_t u = (int64_t)blockIdx.x * kDownUnits + mine;
  if (u < units) {
    const int t = (int)(u / a.D), d = (int)(u - (int64_t)t * a.D);
    for (int j = j0; j < j1; ++j) {
      const int e = __ldcg(a.ids + t * a.k + j);
      if ((unsigned)e >= (unsigned)a.E) continue;
      const uint16_t* w = a.W2t + ((int64_t)e * a.D + d) * a.N1;
      for (int c = lane * 64; c < a.N1; c += 32 * 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(w + c));
    }
  }
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  for (int64_t base = (int64_t)blockIdx.x * kDownUnits, n = 0; base < units;
       base += (int64_t)gridDim.x * kDownUnits, ++n) {
    u = base + mine;
    float y = 0.0f;
    const int t = (int)(u / a.D), d = (int)(u - (int64_t)t * a.D);
    if (u < units)
      for (int j = j0; j < j1; j += 2) {  // two experts' rows at a time, their loads in flight together
        const uint16_t* w[2];
        const float* h = a.h + (int64_t)(t * a.k + j) * a.N1;
        float s[2] = {0.0f, 0.0f}, f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int e = j + i < j1 ? a.ids[t * a.k + j + i] : -1;
          const bool on = (unsigned)e < (unsigned)a.E;
          w[i] = on ? a.W2t + ((int64_t)e * a.D + d) * a.N1 : nullptr;
          f[i] = on ? a.weights[t * a.k + j + i] : 0.0f;
        }
#pragma unroll 4
        for (int c = lane * 8; c < a.N1; c += 256) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (w[i]) {
              const uint4 v = ld_stream(w[i] + c);
              const float4* p = reinterpret_cast<const float4*>(h + (int64_t)i * a.N1 + c);
              s[i] = dot8f(v, p[0], p[1], s[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (w[i]) y += f[i] * s[i];
      }
    y = warp_add(y);
    if (lane == 0) sums[n & 1][mine][part] = y;
    __syncthreads();  // the other half of `sums` is free again: its readers passed this barrier
    if (part == 0 && lane == 0 && u < units) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kDownSplit; ++i) s += sums[n & 1][mine][i];
      a.Y[(int64_t)t * a.D + d] = (uint16_t)(pack2(s, 0.0f) & 0xffffu);
    }
  }
}

}  // namespace moe
}  // namespace cusync
