// What a linear layer's backward pass does besides its products: the gradient at the
// pre-activations, the bias's, and 8-bit rows as bf16.  Bound by memory, as the norm.
#pragma once
#include "lin_math.cuh"

namespace cusync {
namespace lin {

struct DzArgs {
  const uint16_t* dY;
  const uint8_t *Zq, *Ze;
  uint16_t* dZ;         // [M, parts * N], times the fractions of Xs where there are; or NULL (dY itself is dZ)
  const float* Xs;      // 8-bit X, where dWt is wanted: its scales,
  const uint4* q;       // its values [M, K]
  uint4* x;             // and in bf16, times the powers of two in Xs
  int64_t pieces;       // M * K / 16
  int32_t row_pieces;   // K / 16
  int64_t x_pitch, dz_pitch;  // columns from a row of x, of dZ to the next
  float* part;    // [parts][parts of a row * N] sums of dZ over a block's rows, or NULL
  int32_t* err;   // the call's error word, cleared by the call's first kernel
  int64_t M;
  int32_t N, rows;  // rows of a block
  int32_t col_blocks, parts;
};

constexpr int kDzCols = 256;
constexpr int kUnpackPieces = 8;  // of 16 values a thread

// dZ = act'(z) dY from the checkpoint, and the sums over rows that dbias is made of (before
// dZ's rounding).  A lane takes 8 columns, a warp every eighth row of the block's, two rows at a time: with
// four, and two blocks an SM for their registers, the sums alone took 26 us where they take 20.6 (SwiGLU, 4096 x
// 3584: 89 MB, 13.1 us at HBM's rate).
//
// dWt of 8-bit rows X = s q, s = f 2^e with f in [1, 2), is the product of f dZ with 2^e q: the latter is exact in
// bf16, so that there is one rounding, f dZ's, as with X in bf16 (of dZ with s q rounded to bf16 there would be
// two).  dX is the product of the same f dZ, its rows divided by f.  The blocks behind those of dZ write 2^e q.
template <int ACT>
__global__ void __launch_bounds__(256, 3) dz_kernel(const DzArgs a) {
  constexpr int G = ACT == ACT_SWIGLU ? 2 : 1;
  __shared__ float sums[8][kDzCols + 8];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  if (a.err && blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int own = blockIdx.x / a.col_blocks, col_block = blockIdx.x - own * a.col_blocks;
  if (own >= a.parts) {
    const int64_t b = (int64_t)blockIdx.x - (int64_t)a.parts * a.col_blocks, i0 = b * 256 * kUnpackPieces + threadIdx.x;
    uint4 v[kUnpackPieces];
#pragma unroll
    for (int k = 0; k < kUnpackPieces; ++k)
      if (i0 + k * 256 < a.pieces) v[k] = a.q[i0 + k * 256];
#pragma unroll
    for (int k = 0; k < kUnpackPieces; ++k) {
      if (i0 + k * 256 >= a.pieces) break;
      float f[2][8];
      const int64_t i = i0 + k * 256, row = i / a.row_pieces;
      const float power = scale_power(a.Xs[row]);
      unpack_e4m3(v[k].x, f[0]);
      unpack_e4m3(v[k].y, f[0] + 4);
      unpack_e4m3(v[k].z, f[1]);
      unpack_e4m3(v[k].w, f[1] + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[0][j] *= power, f[1][j] *= power;
      uint4* out = a.x + (row * a.x_pitch + (i - row * a.row_pieces) * 16) / 8;
      out[0] = pack8(f[0]);
      out[1] = pack8(f[1]);
    }
    return;
  }
  const int c = col_block * kDzCols + lane * 8;
  const int blocks = (a.N + kBlock - 1) / kBlock;
  const int64_t r0 = (int64_t)own * a.rows, end = min(r0 + a.rows, a.M);
  float acc[G][8];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[g][j] = 0.0f;
  if (c < a.N) {
#pragma unroll 2
    for (int64_t r = r0 + warp; r < end; r += 8) {
      float dy[8], z[G][8];
      unpack8(*reinterpret_cast<const uint4*>(a.dY + r * a.N + c), dy);
      if (ACT != ACT_NONE) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint2 q = *reinterpret_cast<const uint2*>(a.Zq + (r * G + g) * a.N + c);
          const float e = exponent_value(a.Ze[(r * G + g) * blocks + c / kBlock]);
          unpack_e4m3(q.x, z[g]);
          unpack_e4m3(q.y, z[g] + 4);
#pragma unroll
          for (int j = 0; j < 8; ++j) z[g][j] *= e;
        }
      }
      float dz[G][8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (ACT == ACT_NONE) {
          dz[0][j] = dy[j];
        } else if (ACT == ACT_RELU) {
          // NaN, which a checkpoint holds of infinities too, stays NaN, as it does in the other slopes
          dz[0][j] = z[0][j] <= 0.0f ? 0.0f : fmaf(z[0][j], 0.0f, dy[j]);
        } else if (ACT == ACT_GELU) {
          const float x = z[0][j], sg = gelu_gate(x), h = x * sg;
          // far out, where the sigmoid is 0 or 1, the square must not become an infinity
          const float x2 = fminf(x * x, 1e30f);
          dz[0][j] = dy[j] * (sg + h * (1.0f - sg) * 2.0f * kGeluC * (1.0f + 3.0f * 0.044715f * x2));
        } else {
          const float x = z[0][j], u = z[G - 1][j], sg = sigmoid_fast(x), h = x * sg;
          dz[0][j] = dy[j] * u * (sg + h * (1.0f - sg));
          dz[G - 1][j] = dy[j] * h;
        }
#pragma unroll
        for (int g = 0; g < G; ++g) acc[g][j] += dz[g][j];
      }
      if (a.dZ) {
        const float f = a.Xs ? scale_fraction(a.Xs[r]) : 1.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
          for (int j = 0; j < 8; ++j) dz[g][j] *= f;
          *reinterpret_cast<uint4*>(a.dZ + r * a.dz_pitch + g * a.N + c) = pack8(dz[g]);
        }
      }
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[warp][lane * 8 + j] = acc[g][j];
    __syncthreads();
    const int col = col_block * kDzCols + threadIdx.x;
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += sums[w][threadIdx.x];
    if (col < a.N) a.part[((int64_t)own * G + g) * a.N + col] = t;
  }
}

}  // namespace lin
}  // namespace cusync
