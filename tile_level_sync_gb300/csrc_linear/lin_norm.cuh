// The norm and its gradient, and 8-bit rows.  Bound by memory: every tensor is read or written
// once, in 16-byte pieces; sums are in 32 bits and of a fixed order.
#pragma once
#include "lin_math.cuh"

namespace cusync {
namespace lin {

// Sum and maximum over a block's threads, in every thread; one call in a kernel's loop needs
// the other of the two buffers next.
__device__ __forceinline__ float2 block_sum_max(float sum, float most, float2* buf) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (warps == 1) return make_float2(sum, most);
  if (lane == 0) buf[threadIdx.x >> 5] = make_float2(sum, most);
  __syncthreads();
  const float2 v = lane < warps ? buf[lane] : make_float2(0.0f, 0.0f);
  sum = v.x;
  most = v.y;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  return make_float2(sum, most);
}
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* buf) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (warps == 1) return make_float2(a, b);
  if (lane == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  const float2 v = lane < warps ? buf[lane] : make_float2(0.0f, 0.0f);
  a = v.x;
  b = v.y;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  return make_float2(a, b);
}

struct NormArgs {
  const uint4 *X, *R, *w;
  uint4 *S, *Y;
  uint2* Q;
  float* Qs;
  int64_t M;
  int32_t vecs;  // D / 8
  int32_t rms;
  float eps, inv_d;
};

// Squares of a row's values leave fp32's range before the values do.  Where the mean of the squares
// plus eps, v, is outside of what follows, the row is taken times this power of two instead.
__device__ __forceinline__ bool squares_fit(float v) { return v >= 0x1p-100f && v <= 0x1p120f; }
__device__ __forceinline__ float square_scale(float v) { return v > 1.0f ? 0x1p-70f : 0x1p70f; }

// A block takes a row and keeps it in registers: V pieces of 8 columns a thread.  The sum of
// squares and the largest |S w| come out of one pass, as the row's factor r = 1 / sqrt(mean + eps)
// is common to all: max |y| = r max |S w|.
template <int V, int T>
__global__ void __launch_bounds__(T) norm_kernel(const NormArgs a) {
  __shared__ float2 buf[2][32];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int64_t base = (int64_t)blockIdx.x * a.vecs;
  float t[V][8];
  uint4 x[V], r[V], g[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = threadIdx.x + v * blockDim.x;
    x[v] = r[v] = g[v] = make_uint4(0, 0, 0, 0);
    if (i < a.vecs) {
      x[v] = a.X[base + i];
      if (a.R) r[v] = a.R[base + i];
      if (a.rms) g[v] = a.w[i];
    }
  }
  float sum = 0.0f, most = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = threadIdx.x + v * blockDim.x;
    unpack8(x[v], t[v]);
    if (a.R) {
      float f[8];
      unpack8(r[v], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) t[v][j] += f[j];
    }
    if (a.S && i < a.vecs) a.S[base + i] = pack8(t[v]);
    if (a.rms) {
      float w[8];
      unpack8(g[v], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum = fmaf(t[v][j], t[v][j], sum);
        most = fmaxf(most, finite_abs(t[v][j] * w[j]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) most = fmaxf(most, finite_abs(t[v][j]));
    }
  }
  float2 all = block_sum_max(sum, most, buf[0]);
  float f = 1.0f;
  if (a.rms) {
    float square = all.x * a.inv_d + a.eps, c = 1.0f;
    if (!squares_fit(square)) {
      c = square_scale(square);
      sum = most = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float w[8];
        unpack8(g[v], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = t[v][j] * c;
          sum = fmaf(x, x, sum);
          most = fmaxf(most, finite_abs(x * w[j]));
        }
      }
      all = block_sum_max(sum, most, buf[1]);
      square = all.x * a.inv_d + a.eps * c * c;
    }
    f = 1.0f / sqrtf(square);
    all.y *= f;
    f *= c;
  }
  // the factor is NaN or 0 where the row holds NaN or infinities: nothing finite is left, or zeros
  const float scale = fmaxf(finite_abs(all.y) * (1.0f / kE4m3Max), kLeastScale);
  const float inv = 1.0f / scale;
  if (a.Q && threadIdx.x == 0) a.Qs[blockIdx.x] = scale;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = threadIdx.x + v * blockDim.x;
    if (i >= a.vecs) continue;
    if (a.rms) {
      float w[8];
      unpack8(g[v], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) t[v][j] = t[v][j] * f * w[j];
    }
    if (a.Y) a.Y[base + i] = pack8(t[v]);
    if (a.Q) {
#pragma unroll
      for (int j = 0; j < 8; ++j) t[v][j] = no_inf(t[v][j]) * inv;
      a.Q[base + i] = make_uint2(pack_e4m3(t[v][0], t[v][1], t[v][2], t[v][3]),
                                 pack_e4m3(t[v][4], t[v][5], t[v][6], t[v][7]));
    }
  }
}

struct NormGradArgs {
  const uint4 *S, *w, *dY, *dS;
  uint4* dX;
  float* part;   // [blocks][D] sums of dY S r over a block's rows, or NULL
  int32_t* err;
  int64_t M;
  int32_t vecs;
  int32_t stages;  // rows of the ring
  float eps, inv_d;
};

constexpr int kNormStages = 8;
constexpr uint64_t kNormWaitNs = 1000000000ull;
constexpr uint32_t kNormErrWait = 3u << 24;

// dX = r (g - S r mean(g S r)) + dS with g = w dY; a block takes rows blockIdx.x, + gridDim.x, ...
// and keeps its columns' share of dw in registers.  A row's tensors come by bulk copies into a ring of
// `stages` rows, so that the next rows are under way while this one waits for its sums: the same
// kernel with rows loaded into registers reached 4230 GB/s where this one reaches 6090 (8192 x 8192, dS added).
template <int V, int T>
__global__ void __launch_bounds__(T, 1) norm_grad_kernel(const NormGradArgs a) {
  extern __shared__ __align__(128) uint4 rows[];
  __shared__ float2 buf[4][32];
  __shared__ uint64_t full[kNormStages];
  const int tensors = a.dS ? 3 : 2, stages = a.stages;
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) ptx::mbar_init(&full[i], 1);
    ptx::mbar_init_fence();
  }
  __syncthreads();
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  const uint32_t bytes = (uint32_t)a.vecs * 16;
  auto fetch = [&](int64_t row, int st) {  // one thread
    if (row >= a.M) return;
    uint4* to = rows + (int64_t)st * tensors * a.vecs;
    ptx::mbar_arrive_expect_tx(&full[st], tensors * bytes);
    ptx::bulk_load(to, a.S + row * a.vecs, bytes, &full[st]);
    ptx::bulk_load(to + a.vecs, a.dY + row * a.vecs, bytes, &full[st]);
    if (a.dS) ptx::bulk_load(to + 2 * a.vecs, a.dS + row * a.vecs, bytes, &full[st]);
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < stages; ++i) fetch(blockIdx.x + (int64_t)i * gridDim.x, i);
  float dw[V][8];
  uint4 wv[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = threadIdx.x + v * blockDim.x;
    wv[v] = i < a.vecs ? a.w[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[v][j] = 0.0f;
  }
  int turn = 0, st = 0;
  uint32_t par = 0;
  bool ok = true;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
    // after a wait that gave up: on with what is there
    if (ok && !ptx::mbar_wait_bounded(&full[st], par, kNormWaitNs)) {
      ok = false;
      *a.err = (int32_t)kNormErrWait;
    }
    const uint4 *x = rows + (int64_t)st * tensors * a.vecs, *y = x + a.vecs, *s = y + a.vecs;
    float squares = 0.0f, dots = 0.0f;
    auto sums = [&](float c) {
      squares = dots = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        if (i >= a.vecs) continue;
        float fx[8], fy[8], fw[8];
        unpack8(x[i], fx);
        unpack8(y[i], fy);
        unpack8(wv[v], fw);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xc = fx[j] * c;
          squares = fmaf(xc, xc, squares);
          dots = fmaf(fy[j] * fw[j], xc, dots);
        }
      }
    };
    sums(1.0f);
    float2 all = block_sum2(squares, dots, buf[turn]);
    // behind that barrier every thread is done with the row before: its place takes the row `stages` further
    if (threadIdx.x == 0 && stages > 1 && row >= gridDim.x) {
      const int before = st ? st - 1 : stages - 1;
      fetch(row + (int64_t)(stages - 1) * gridDim.x, before);
    }
    float square = all.x * a.inv_d + a.eps, c = 1.0f;
    if (!squares_fit(square)) {
      c = square_scale(square);
      sums(c);
      all = block_sum2(squares, dots, buf[2 + turn]);
      square = all.x * a.inv_d + a.eps * c * c;
    }
    const float rc = 1.0f / sqrtf(square), mean = all.y * a.inv_d * rc, r = rc * c;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = threadIdx.x + v * blockDim.x;
      if (i >= a.vecs) continue;
      float fx[8], fy[8], fw[8], fs[8];
      unpack8(x[i], fx);
      unpack8(y[i], fy);
      unpack8(wv[v], fw);
      unpack8(a.dS ? s[i] : make_uint4(0, 0, 0, 0), fs);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = fx[j] * r;
        dw[v][j] = fmaf(fy[j], xh, dw[v][j]);
        fs[j] += r * (fy[j] * fw[j] - xh * mean);
      }
      a.dX[row * a.vecs + i] = pack8(fs);
    }
    if (stages == 1) {
      __syncthreads();
      if (threadIdx.x == 0) fetch(row + gridDim.x, 0);
    }
    if (++st == stages) {
      st = 0;
      par ^= 1;
    }
  }
  if (a.part) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = threadIdx.x + v * blockDim.x;
      if (i >= a.vecs) continue;
      float4* out = reinterpret_cast<float4*>(a.part) + ((int64_t)blockIdx.x * a.vecs + i) * 2;
      out[0] = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
      out[1] = make_float4(dw[v][4], dw[v][5], dw[v][6], dw[v][7]);
    }
  }
}

}  // namespace lin
}  // namespace cusync
