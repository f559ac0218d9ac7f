// The norm and its gradient, and 8-bit rows.  Bound by memory: every tensor is read or written
// once, in 16-byte pieces; sums are in 32 bits and of a fixed order.
//
// A row of at most kWarpVecs pieces of 8 columns is a warp's, a longer one a block's; each thread keeps up to four
// pieces of it in registers.  (A block for each row of 256 columns took 17.4 us where warps take 5.9, 16384 rows of the
// norm with residual and 8 bits out; the gradient of such rows 21.5 and 13.0, of 4096 rows of 1024 20.4 and 10.5.)
#pragma once
#include "lin_math.cuh"

namespace cusync {
namespace lin {

constexpr int kWarpVecs = 128;  // 1024 columns
constexpr int kRowWarps = 8;    // of a block whose warps take rows

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// The sum of a, and the sum or maximum of b, over the threads that share a row, in each of them.
struct WarpRow {
  static constexpr bool kBlock = false;
  __device__ __forceinline__ void sync() const { __syncwarp(); }
  template <bool MAX>
  __device__ __forceinline__ float2 reduce(float a, float b, int) const {
    return make_float2(warp_sum(a), MAX ? warp_max(b) : warp_sum(b));
  }
};
struct BlockRow {
  static constexpr bool kBlock = true;
  __device__ __forceinline__ void sync() const { __syncthreads(); }
  float2 (*buf)[32];  // one call needs another buffer than the one before it
  template <bool MAX>
  __device__ __forceinline__ float2 reduce(float a, float b, int turn) const {
    const float2 w = WarpRow().reduce<MAX>(a, b, 0);
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) buf[turn][threadIdx.x >> 5] = w;
    __syncthreads();
    const float2 v = lane < warps ? buf[turn][lane] : make_float2(0.0f, 0.0f);
    return WarpRow().reduce<MAX>(v.x, v.y, 0);
  }
};

// Squares of a row's values leave fp32's range before the values do.  Where the mean of the squares
// plus eps, v, is outside of what follows, the row is taken times this power of two instead: 2^15 squares of values
// below 2^128 then add up to less than 2^111, and a square of 2^-133 alone among as many columns has a mean of 2^-121.
__device__ __forceinline__ bool squares_fit(float v) { return v >= 0x1p-100f && v <= 0x1p120f; }
// The power's root.  A row takes it and so does its factor r, each of which stays within 32 bits then: r alone is beyond
// them for rows below 2^-128.
__device__ __forceinline__ float square_scale(float v) { return v > 1.0f ? 0x1p-40f : 0x1p40f; }

// Whether a row's max |y| is r times `most`, its max |S w| in 32 bits: where neither is infinite and the product has all of
// its bits, or where it is 0, below 2^-149, and y so small that the least scale is the row's (rows of zeros: 8192 x 8192 of
// them took 143 us as odd rows, and 48 so).
__device__ __forceinline__ bool product_fits(float most, float r) {
  return most <= kFloatMax && most * r <= kFloatMax && (most >= kLeastScale || (most == 0.0f && r <= 0x1p32f));
}

constexpr uint32_t kOnes = 0x3f803f80u;  // two bf16 ones

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

// y of a row whose squares, or whose products S w, do not fit, in t's place (S on entry); returns the largest finite |y|.  A
// call of its own, with t in memory, so that the kernels keep their registers: in line it cost 8192 x 8192 71 us and more
// where this takes 68.7.
template <int V, typename Row>
__device__ __noinline__ float norm_odd_row(float* t, const uint4* weights, int vecs, int i0, int step, float square, float eps,
                                           float inv_d, const Row& threads) {
  const float c = squares_fit(square) ? 1.0f : square_scale(square);
  float sum = 0.0f, most = 0.0f;
#pragma unroll 1
  for (int i = 0; i < 8 * V; ++i) {
    const float xc = t[i] * c * c;
    sum = fmaf(xc, xc, sum);
  }
  sum = threads.template reduce<true>(sum, 0.0f, 1).x;
  const float f = 1.0f / sqrtf(sum * inv_d + eps * (c * c) * (c * c)) * c;
#pragma unroll 1
  for (int v = 0; v < V; ++v) {
    const int at = i0 + v * step;
    float w[8];
    unpack8(at < vecs ? weights[at] : make_uint4(0, 0, 0, 0), w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float y = t[8 * v + j] * c * f * w[j];
      t[8 * v + j] = y;
      most = fmaxf(most, finite_abs(y));
    }
  }
  return threads.template reduce<true>(0.0f, most, 0).y;
}

// One row by the threads i0, i0 + step, ...: V pieces each.  The sum of squares and the largest |S w| come
// out of one pass, as the row's factor r = 1 / sqrt(mean + eps) is common to all: max |y| = r max |S w|.
template <int V, typename Row>
__device__ __forceinline__ void norm_row(const NormArgs& a, int64_t row, int i0, int step, const Row& threads) {
  const int64_t base = row * a.vecs;
  float t[V][8];
  uint4 x[V], r[V], g[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = i0 + v * step;
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
    const int i = i0 + v * step;
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
        most = fmaxf(most, fabsf(t[v][j] * w[j]));  // passes a NaN by, keeps infinities
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) most = fmaxf(most, finite_abs(t[v][j]));
    }
  }
  float2 all = threads.template reduce<true>(sum, most, 0);
  float f = 1.0f;
  if (a.rms) {
    const float square = all.x * a.inv_d + a.eps;
    f = 1.0f / sqrtf(square);
    if (!squares_fit(square) || (a.Q && !product_fits(all.y, f))) {
      float y[V * 8];
#pragma unroll
      for (int i = 0; i < 8 * V; ++i) y[i] = t[i / 8][i % 8];
      all.y = norm_odd_row<V>(y, a.w, a.vecs, i0, step, square, a.eps, a.inv_d, threads);
      f = 1.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        g[v] = make_uint4(kOnes, kOnes, kOnes, kOnes);
#pragma unroll
        for (int j = 0; j < 8; ++j) t[v][j] = y[8 * v + j];
      }
    }
    all.y *= f;
  }
  // the factor is NaN or 0 where the row holds NaN or infinities: nothing finite is left, or zeros
  const float scale = fmaxf(finite_abs(all.y) * (1.0f / kE4m3Max), kLeastScale);
  const float inv = 1.0f / scale;
  if (a.Q && i0 == 0) a.Qs[row] = scale;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = i0 + v * step;
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

// Blocks an SM as their loads need: with fewer, 8192 x 8192 in bf16 took 55 us instead of 46, 4096 x 3584 15.1 instead of 14.1.
template <int V, int T>
__global__ void __launch_bounds__(T, T > 256 ? 1 : V == 4 ? 4 : V == 2 ? 6 : 8) norm_block_kernel(const NormArgs a) {
  __shared__ float2 buf[2][32];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  norm_row<V>(a, blockIdx.x, threadIdx.x, blockDim.x, BlockRow{buf});
}
template <int V>
__global__ void __launch_bounds__(kRowWarps * 32) norm_warp_kernel(const NormArgs a) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int64_t row = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (row < a.M) norm_row<V>(a, row, threadIdx.x & 31, 32, WarpRow());
}

struct NormGradArgs {
  const uint4 *S, *w, *dY, *dS;
  uint4* dX;
  float* part;   // [blocks][D] sums of dY S r over a block's rows, or NULL
  int32_t* err;
  int64_t M;
  int32_t vecs;
  int32_t stages;  // rows of a ring
  float eps, inv_d;
};

constexpr int kNormStages = 8;
constexpr uint64_t kNormWaitNs = 1000000000ull;
constexpr uint32_t kNormErrWait = 3u << 24;

// dX = r (g - S r mean(g S r)) + dS with g = w dY.  A warp or a block takes rows first, first + stride, ... and keeps
// its columns' share of dw in registers.  A row's tensors come by bulk copies into a ring of `stages` rows, so that the
// next rows are under way while this one waits for its sums: with rows loaded into registers alone 8192 x 8192 (dS
// added) took 127 us, with the ring 82 (6.5 TB/s).  Where the ring holds three rows or fewer, a row's place is refilled as
// soon as it is read, at the price of a barrier (2000 x 12288: 39.0 us, 43.2 with the row after it).  Four pieces a
// thread, rows above 16384 columns, leave dS out of the ring, which would hold one row with it (2000 x 20480: 131 us
// with it and 120 without; 112 now).
template <int V, typename Row>
__device__ __forceinline__ void norm_grad_rows(const NormGradArgs& a, int64_t first, int64_t stride, int i0, int step,
                                               const Row& threads, uint4* ring, uint64_t* full, float (&dw)[V][8]) {
  const int stages = a.stages;
  const uint32_t bytes = (uint32_t)a.vecs * 16;
  constexpr bool kDirect = V == 4 && Row::kBlock;  // dS
  const int tensors = a.dS && !kDirect ? 3 : 2;
  bool ok = true;
  auto fetch = [&](int64_t row, int st) {  // one thread
    if (row >= a.M || !ok) return;
    uint4* to = ring + (int64_t)st * tensors * a.vecs;
    ptx::mbar_arrive_expect_tx(&full[st], tensors * bytes);
    ptx::bulk_load(to, a.S + row * a.vecs, bytes, &full[st]);
    ptx::bulk_load(to + a.vecs, a.dY + row * a.vecs, bytes, &full[st]);
    if (a.dS && !kDirect) ptx::bulk_load(to + 2 * a.vecs, a.dS + row * a.vecs, bytes, &full[st]);
  };
  if (i0 == 0)
    for (int i = 0; i < stages; ++i) fetch(first + i * stride, i);
  uint4 wv[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = i0 + v * step;
    wv[v] = i < a.vecs ? a.w[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[v][j] = 0.0f;
  }
  int turn = 0, st = 0;
  uint32_t par = 0;
  for (int64_t row = first; row < a.M; row += stride, turn ^= 1) {
    uint4 s[kDirect ? V : 1];
    if (kDirect) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int i = i0 + v * step;
        s[kDirect ? v : 0] = a.dS && i < a.vecs ? a.dS[row * a.vecs + i] : make_uint4(0, 0, 0, 0);
      }
    }
    // after a wait that gave up: on with what is there.  The thread that copies asks for no more rows and waits, with a limit
    // again, for those that it has asked for: no block ends with copies into its memory under way.
    if (ok && !ptx::mbar_wait_bounded(&full[st], par, kNormWaitNs)) {
      ok = false;
      *a.err = (int32_t)kNormErrWait;
      const int asked = stages > 3 && row != first ? stages - 1 : stages;  // the row before's place is free
      if (i0 == 0)
        for (int i = 0, at = st; i < asked && row + i * stride < a.M; ++i) {
          ptx::mbar_wait_bounded(&full[at], at < st ? par ^ 1 : par, kNormWaitNs);
          if (++at == stages) at = 0;
        }
    }
    const uint4 *x = ring + (int64_t)st * tensors * a.vecs, *y = x + a.vecs;
    float squares = 0.0f, dots = 0.0f;
    auto sums = [&](float c) {
      squares = dots = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int i = i0 + v * step;
        if (i >= a.vecs) continue;
        float fx[8], fy[8], fw[8];
        unpack8(x[i], fx);
        unpack8(y[i], fy);
        unpack8(wv[v], fw);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xc = fx[j] * c * c;
          squares = fmaf(xc, xc, squares);
          dots = fmaf(fy[j] * fw[j], xc, dots);
        }
      }
    };
    sums(1.0f);
    float2 all = threads.template reduce<false>(squares, dots, turn);
    // behind these sums every thread is done with the row before: its place takes the row `stages` further.  A block's
    // sums meet at a barrier; a warp's shuffles order no memory.
    if (!Row::kBlock) threads.sync();
    if (i0 == 0 && stages > 3 && row != first) fetch(row + (stages - 1) * stride, st ? st - 1 : stages - 1);
    float square = all.x * a.inv_d + a.eps, c = 1.0f;
    if (!squares_fit(square)) {
      c = square_scale(square);
      sums(c);
      all = threads.template reduce<false>(squares, dots, 2 + turn);
      square = all.x * a.inv_d + a.eps * (c * c) * (c * c);
    }
    const float rc = 1.0f / sqrtf(square), mean = all.y * a.inv_d * rc, r = rc * c;
    auto store = [&](float c) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int i = i0 + v * step;
        if (i >= a.vecs) continue;
        float fx[8], fy[8], fw[8], fs[8];
        unpack8(x[i], fx);
        unpack8(y[i], fy);
        unpack8(wv[v], fw);
        unpack8(kDirect ? s[kDirect ? v : 0] : a.dS ? y[a.vecs + i] : make_uint4(0, 0, 0, 0), fs);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = fx[j] * c * r;
          dw[v][j] = fmaf(fy[j], xh, dw[v][j]);
          fs[j] += r * ((fy[j] * fw[j] - xh * mean) * c);
        }
        a.dX[row * a.vecs + i] = pack8(fs);
      }
    };
    if (c == 1.0f) store(1.0f);
    else store(c);
    if (stages <= 3) {
      threads.sync();
      if (i0 == 0) fetch(row + stages * stride, st);
    }
    if (++st == stages) {
      st = 0;
      par ^= 1;
    }
  }
}

template <int V, int T, int PER_SM>
__global__ void __launch_bounds__(T, PER_SM) norm_grad_block_kernel(const NormGradArgs a) {
  extern __shared__ __align__(128) uint4 rows[];
  __shared__ float2 buf[4][32];
  __shared__ uint64_t full[kNormStages];
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) ptx::mbar_init(&full[i], 1);
    ptx::mbar_init_fence();
  }
  __syncthreads();
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  float dw[V][8];
  norm_grad_rows<V>(a, blockIdx.x, gridDim.x, threadIdx.x, blockDim.x, BlockRow{buf}, rows, full, dw);
  if (!a.part) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = threadIdx.x + v * blockDim.x;
    if (i >= a.vecs) continue;
    float4* out = reinterpret_cast<float4*>(a.part) + ((int64_t)blockIdx.x * a.vecs + i) * 2;
    out[0] = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
    out[1] = make_float4(dw[v][4], dw[v][5], dw[v][6], dw[v][7]);
  }
}

// Each warp has a ring of its own; the warps' shares of dw are added in their order.
template <int V>
__global__ void __launch_bounds__(kRowWarps * 32) norm_grad_warp_kernel(const NormGradArgs a) {
  extern __shared__ __align__(128) uint4 rows[];
  __shared__ uint64_t full[kRowWarps][kNormStages];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
    for (int i = 0; i < a.stages; ++i) ptx::mbar_init(&full[warp][i], 1);
    ptx::mbar_init_fence();
  }
  __syncthreads();
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  float dw[V][8];
  norm_grad_rows<V>(a, (int64_t)blockIdx.x * kRowWarps + warp, (int64_t)gridDim.x * kRowWarps, lane, 32, WarpRow(),
                    rows + (int64_t)warp * a.stages * (a.dS ? 3 : 2) * a.vecs, full[warp], dw);
  if (!a.part) return;
  __syncthreads();  // the rings take [warps][D] sums
  float* sums = reinterpret_cast<float*>(rows);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = lane + v * 32;
    if (i >= a.vecs) continue;
    float4* out = reinterpret_cast<float4*>(sums) + (warp * a.vecs + i) * 2;
    out[0] = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
    out[1] = make_float4(dw[v][4], dw[v][5], dw[v][6], dw[v][7]);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 8 * a.vecs; c += kRowWarps * 32) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) s += sums[w * 8 * a.vecs + c];
    a.part[(int64_t)blockIdx.x * 8 * a.vecs + c] = s;
  }
}

}  // namespace lin
}  // namespace cusync
