// Roundings, 8-bit forms and activations that the norm's and the linear layer's kernels share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../csrc/ptx.cuh"

namespace cusync {
namespace ptx {

// `bytes` (a multiple of 16) from global to shared memory, both 16-byte aligned; completes on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

}  // namespace ptx

namespace lin {

constexpr float kE4m3Max = 448.0f;
constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126: its reciprocal is finite
constexpr float kFloatMax = 3.402823466e38f;
constexpr int kBlock = 32;                      // columns that share an exponent in a checkpoint

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
// |v|, or 0 where it is infinite or NaN
__device__ __forceinline__ float finite_abs(float v) { return fabsf(v) <= kFloatMax ? fabsf(v) : 0.0f; }
// Infinities as NaN, which e4m3 has; the conversion itself would make them 448.
__device__ __forceinline__ float no_inf(float v) { return fabsf(v) <= kFloatMax ? v : __uint_as_float(0x7fffffffu); }
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
__device__ __forceinline__ void unpack_e4m3(uint32_t v, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v >> (16 * i)), __NV_E4M3);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

// A checkpoint block's exponent from its largest finite magnitude: 448 = 1.75 * 2^8, so a fraction up to
// 1.75 needs eight binades less than the magnitude's own.
__device__ __forceinline__ uint32_t block_exponent(float most) {
  const uint32_t bits = __float_as_uint(most);
  const int e = (int)(bits >> 23) - 8 + ((bits & 0x007fffffu) > 0x00600000u);
  return (uint32_t)max(e, 1);
}
__device__ __forceinline__ float exponent_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }
__device__ __forceinline__ float exponent_value(uint32_t e) { return __uint_as_float(e << 23); }

// 2^x and 1 / x to 2 ulp, one instruction each (the full functions cost the forward epilogue 41.6 us instead of 39.4,
// 4096 x 1024 x 4096 with GeLU); 0 below 2^-126, so that a gate below -87.3 counts as 0 where its silu is -1e-36 or nearer
// to 0, and infinity above fp32's range
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
// A row's scale as f * +-2^e with f in [1, 2): f, and +-2^e (infinities and NaN whole; below 2^-126: 0).
__device__ __forceinline__ float scale_fraction(float s) {
  return __uint_as_float((__float_as_uint(s) & 0x007fffffu) | 0x3f800000u);
}
__device__ __forceinline__ float scale_power(float s) {
  return fabsf(s) <= kFloatMax ? __uint_as_float(__float_as_uint(s) & 0xff800000u) : s;
}

// 1 / (1 + e^-x)
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp_fast(1.0f + exp2_fast(x * -kLog2e)); }
// GeLU_tanh(z) = z sigmoid(2 c (z + 0.044715 z^3)); the sigmoid's argument as z (a + b z^2)
__device__ __forceinline__ float gelu_gate(float z) {
  constexpr float a = -2.0f * kGeluC * kLog2e, b = 0.044715f * a;
  return rcp_fast(1.0f + exp2_fast(z * fmaf(z * z, b, a)));
}

enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_SWIGLU = 3 };

__device__ __forceinline__ float activate(float z, int act) {
  // a NaN passes the comparison
  return act == ACT_RELU ? (z < 0.0f ? 0.0f : z) : act == ACT_GELU ? z * gelu_gate(z) : z;
}

// out [cols] bf16 = sums of part [rows][cols] over its rows.  A block takes 32 columns: 8 threads of
// four, 32 groups of rows; the groups' sums are added in order.
static __global__ void __launch_bounds__(256) column_sum_kernel(const float* part, int32_t rows, int32_t cols, uint16_t* out) {
  __shared__ float4 sums[32][8];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int piece = threadIdx.x & 7, group = threadIdx.x >> 3;
  const int c = blockIdx.x * 32 + piece * 4;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < cols) {
    for (int r0 = group; r0 < rows; r0 += 32 * 8) {  // eight loads at a time, whatever is left
      float4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        v[k] = r0 + 32 * k < rows ? *reinterpret_cast<const float4*>(part + (int64_t)(r0 + 32 * k) * cols + c)
                                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s.x += v[k].x;
        s.y += v[k].y;
        s.z += v[k].z;
        s.w += v[k].w;
      }
    }
  }
  sums[group][piece] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int col = blockIdx.x * 32 + threadIdx.x;
    float t = 0.0f;
#pragma unroll
    for (int g = 0; g < 32; ++g) t += reinterpret_cast<const float*>(&sums[g][0])[threadIdx.x];
    if (col < cols) out[col] = __bfloat16_as_ushort(__float2bfloat16_rn(t));
  }
}

}  // namespace lin
}  // namespace cusync
