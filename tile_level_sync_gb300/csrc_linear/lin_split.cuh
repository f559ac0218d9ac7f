// The products of a linear layer with few output tiles: a cluster of CTAs for each tile, the
// reduction divided among them.
//
//   mode   A (M: 128 features)          B (N: `cols` tokens)    output row      output column
//   FWD    Wt rows (SwiGLU: 64 gate,    X rows                  token           feature
//          then 64 up rows)
//   DX     Wt along K                   dZ rows                 token           column of X
//   DW     X along K (K: tokens)        dZ along N              row of Wt       column of Wt
//
// A decoding batch reads every weight once and multiplies it with a few tokens: what counts is
// that all SMs stream weights at once.  Weights are the MMA's rows, whose number is fixed, and tokens
// its columns, of which 16 will do.  A tile's reduction is cut into `splits` runs, one for each CTA
// of a cluster; their fp32 sums meet in shared memory: each CTA sends every other one the columns that
// that one finishes, and adds what it gets in the CTAs' order.  The sums are counted by a barrier of the CTA
// that they go to, which waits for them alone.  No partial sum leaves the SMs, and one launch does it all.
//
// What bounds it: HBM while the weights come (59 MB of one token's layer 3584 -> 8192 in 8 us of 12.7, and the same of 48
// tokens' 8192 -> 3584 with SwiGLU in e4m3 of 13.9: traced from the first copy to the last MMA), and 5 us around: the end
// of the kernel before, the first bytes' latency, exchange and finish.  Copying the weights' first stages to the L2
// before the kernel before has ended gained nothing (13.7 us without, 13.9 with, 15.0 with all stages).
//
// Roles: warp 0 copies A, warp 2 copies B, warp 1 owns TMEM and issues the MMAs; then all
// eight warps read the accumulator, exchange and finish.  Every wait is bounded.
#pragma once
#include "lin_gemm.cuh"
#include "lin_plan.h"

namespace cusync {
namespace ptx {

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

}  // namespace ptx

namespace lin {

struct SplitArgs {
  CUtensorMap mA, mB;
  Epilogue e;
  int32_t* err;
  int32_t clear;
  int32_t M, N, K;       // output rows, output columns (SwiGLU: of Y), reduction length
  int32_t b_rows;           // rows of B that are copied: cols, or fewer where there are fewer, a multiple of 8
  int32_t cols, row_tiles;  // MMA columns (output rows) of a tile: 16, 32, 64 or 128; tiles of them
  int32_t splits;        // CTAs of a cluster, at most the reduction's stages
  int32_t stages;        // of the ring
  int32_t apart;         // the sums have room of their own behind the ring, else they take the ring's
  int32_t wideA, wideB;
};

constexpr int kSplitThreads = 256;

template <int MODE, bool E4M3, bool GATED>
__global__ void __launch_bounds__(kSplitThreads) split_kernel(const __grid_constant__ SplitArgs a) {
  constexpr bool kMnA = MODE != FWD, kMnB = MODE == DW;
  constexpr int kElems = E4M3 ? 128 : 64;
  constexpr int kFeatures = GATED ? 64 : 128;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], tfull, drain, came;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int32_t abort_flag;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int splits = a.splits, rank = splits > 1 ? (int)ptx::cluster_ctarank() : 0;
  const uint32_t tmem_cols = a.cols < 32 ? 32 : a.cols;

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    ptx::mbar_init(&tfull, 1);
    ptx::mbar_init(&drain, 1);
    ptx::mbar_init(&came, 1);
    ptx::mbar_init_fence();
    if (splits > 1) ptx::mbar_arrive_expect_tx(&came, a.cols * 128 * 4);
    abort_flag = 0;
    ptx::prefetch_tmap(&a.mA);
    ptx::prefetch_tmap(&a.mB);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&tmem_slot, tmem_cols);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  }
  __syncthreads();
  if (splits > 1) ptx::cluster_arrive();  // this CTA's barriers exist
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);

  const int t = blockIdx.x / splits;
  const int f_first = t / a.row_tiles * kFeatures, r_first = t % a.row_tiles * a.cols;
  const int f0 = span_start(f_first, a.N, kFeatures, kMnA ? 64 : 32), r0 = span_start(r_first, a.M, a.cols, kMnB ? 64 : 1);
  const int nkb = (a.K + kElems - 1) / kElems;
  const int all = (nkb + 1) / 2;  // stages of the whole reduction; this CTA's:
  const int s0 = (int)((int64_t)all * rank / splits), s1 = (int)((int64_t)all * (rank + 1) / splits);
  const int a_bytes = 2 * 128 * 128, b_bytes = 2 * a.b_rows * 128, stage_bytes = split_stage_bytes(a.cols);
  // where a stage's block b begins, and an "along" operand's second chunk of 64 columns
  const int b_step = a.b_rows * 128, chunk = 2 * 64 * 128;

  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  if (a.clear && blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  bool ok = true;

  if (warp == 0 || warp == 2) {
    const bool copies_a = warp == 0;
    const uint64_t pol = ptx::l2_policy_evict_normal();
    const bool one = ptx::elect_one();
    int st = 0, it = 0;
    uint32_t par = 1;
    for (int s = s0; s < s1; ++s, ++it) {
      ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(&empty[st], par, kWaitNs));
      if (!ok || abort_flag) break;
      const int kb = 2 * s;
      const bool half = kb + 1 == nkb;  // the stage's second block holds nothing
      uint8_t* sA = ring + st * stage_bytes;
      uint8_t* sB = sA + a_bytes;
      uint64_t* bar = &full[st];
      if (one && copies_a) {
        const uint32_t as = kMnA || a.wideA || !half ? a_bytes : a_bytes / 2;
        const uint32_t bs = kMnB || a.wideB || !half ? b_bytes : b_bytes / 2;
        ptx::mbar_arrive_expect_tx(bar, as + bs);
        if (kMnA) {
          if (a.wideA) {
            ptx::tma_load_3d(sA, &a.mA, bar, 0, kb * 64, f0 / 64, pol);
          } else {
            ptx::tma_load_2d(sA, &a.mA, bar, f0, kb * 64, pol);
            ptx::tma_load_2d(sA + chunk, &a.mA, bar, f0 + 64, kb * 64, pol);
          }
        } else if (a.wideA) {
          if (GATED) ptx::tma_load_4d(sA, &a.mA, bar, 0, f0, 0, kb, pol);
          else ptx::tma_load_3d(sA, &a.mA, bar, 0, f0, kb, pol);
        } else {
          for (int b = 0; b < (half ? 1 : 2); ++b) {
            if (GATED) ptx::tma_load_3d(sA + b * 16384, &a.mA, bar, (kb + b) * kElems, f0, 0, pol);
            else ptx::tma_load_2d(sA + b * 16384, &a.mA, bar, (kb + b) * kElems, f0, pol);
          }
        }
      }
      if (one && !copies_a) {
        if (kMnB) {
          if (a.wideB) {
            ptx::tma_load_3d(sB, &a.mB, bar, 0, kb * 64, r0 / 64, pol);
          } else {
            ptx::tma_load_2d(sB, &a.mB, bar, r0, kb * 64, pol);
            if (a.cols > 64) ptx::tma_load_2d(sB + chunk, &a.mB, bar, r0 + 64, kb * 64, pol);
          }
        } else if (a.wideB) {
          ptx::tma_load_3d(sB, &a.mB, bar, 0, r0, kb, pol);
        } else {
          for (int b = 0; b < (half ? 1 : 2); ++b)
            ptx::tma_load_2d(sB + b * b_step, &a.mB, bar, (kb + b) * kElems, r0, pol);
        }
      }
      __syncwarp();
      if (++st == a.stages) {
        st = 0;
        par ^= 1;
      }
    }
    if (!ok) abort_flag = 1;
    __syncwarp();
    // after an abort: wait, bounded, for the copies still in flight (both warps' complete on `full`)
    if (abort_flag && copies_a && lane == 0)
      for (int i = it > a.stages ? it - a.stages : 0; i < it; ++i)
        ptx::mbar_wait_bounded(&full[i % a.stages], (i / a.stages) & 1, kWaitNs);
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t ring0 = __shfl_sync(0xffffffffu, ptx::smem_u32(ring), 0);
    const bool one = ptx::elect_one();
    const uint32_t idesc = (E4M3 ? ptx::idesc_e4m3_f32(128, a.cols) : ptx::idesc_bf16_f32(128, a.cols)) |
                           (kMnA ? ptx::kIdescAMn : 0) | (kMnB ? ptx::kIdescBMn : 0);
    int st = 0;
    uint32_t par = 0;
    for (int s = s0; s < s1; ++s) {
      ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(&full[st], par, kWaitNs));
      if (!ok || abort_flag) break;
      ptx::tc_fence_after();
      const uint32_t sA = ring0 + st * stage_bytes, sB = sA + a_bytes;
      const uint64_t dA = kMnA ? ptx::smem_desc_mn128(sA, chunk) : ptx::smem_desc_k128(sA);
      const uint64_t dB = kMnB ? ptx::smem_desc_mn128(sB, chunk) : ptx::smem_desc_k128(sB);
      const int steps = (a.K - 2 * s * kElems + kElems / 4 - 1) / (kElems / 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i >= steps) break;
        if (!one) continue;
        const uint64_t mn = (uint64_t)(i * 2048) >> 4;
        const uint64_t oA = kMnA ? mn : (uint64_t)(i / 4 * 16384 + i % 4 * 32) >> 4;
        const uint64_t oB = kMnB ? mn : (uint64_t)(i / 4 * b_step + i % 4 * 32) >> 4;
        if (E4M3) ptx::umma_e4m3(tmem, dA + oA, dB + oB, idesc, s > s0 || i);
        else ptx::umma_bf16(tmem, dA + oA, dB + oB, idesc, s > s0 || i);
      }
      if (one) ptx::umma_commit(&empty[st]);
      __syncwarp();
      if (++st == a.stages) {
        st = 0;
        par ^= 1;
      }
    }
    if (ok && !abort_flag) {
      if (one) ptx::umma_commit(&tfull);
    } else {
      abort_flag = 1;
      if (one) ptx::umma_commit(&drain);  // MMAs still in flight
      ptx::mbar_wait_bounded(&drain, 0, kWaitNs);
    }
    __syncwarp();
  }

  // ------------------------------------------------------------ exchange
  // A thread finishes the same 8 features of all its tokens: their scales and biases, while the product runs.
  constexpr int kGroups = kFeatures / 8;
  const Epilogue& e = a.e;
  const int group = threadIdx.x % kGroups, c = f0 + group * 8;
  float ws[GATED ? 2 : 1][8], bs[GATED ? 2 : 1][8];
#pragma unroll
  for (int g = 0; g < (GATED ? 2 : 1); ++g) {
#pragma unroll
    for (int j = 0; j < 8; ++j) ws[g][j] = 1.0f, bs[g][j] = 0.0f;
    if (E4M3 && c < a.N) load8(e.Ws + (int64_t)g * a.N + c, ws[g]);
    if (MODE == FWD && e.bias && c < a.N) load8(e.bias + (int64_t)g * a.N + c, bs[g]);
  }
  ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleepy(&tfull, 0, 2 * kWaitNs)) && ok;
  if (!ok) {
    abort_flag = 1;
    *a.err = (int32_t)kErrWait;
  }
  ptx::tc_fence_after();
  const int per = a.cols / splits, shift = 31 - __clz(per);
  float* sums = reinterpret_cast<float*>(ring + (a.apart ? a.stages * stage_bytes : 0));  // [splits][per][128]
  if (splits > 1) {
    ptx::cluster_wait();
    if (!a.apart) {  // every CTA's MMAs have read its ring
      __syncthreads();
      ptx::cluster_sync();
    }
  }
  {
    const int quarter = warp & 3, m = 32 * quarter + lane, width = a.cols / 2, c0 = (warp >> 2) * width;
    const uint32_t d = tmem + ((uint32_t)(32 * quarter) << 16);
    float* mine = sums + rank * per * 128 + m;  // this CTA's sums, wherever they go
    auto put = [&](int n, uint32_t v) {
      const int to = n >> shift;
      if (splits > 1) ptx::st_async_u32(ptx::mapa(mine + (n & (per - 1)) * 128, to), v, ptx::mapa(&came, to));
      else mine[n * 128] = __uint_as_float(v);
    };
    if (width >= 32) {
#pragma unroll 1
      for (int c = c0; c < c0 + width; c += 32) {
        uint32_t v[32];
        ptx::tmem_ld_32x32b_x32(d + c, v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) put(c + i, v[i]);
      }
    } else {
#pragma unroll 1
      for (int c = c0; c < c0 + width; c += 8) {
        uint32_t v[8];
        ptx::tmem_ld_32x32b_x8(d + c, v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) put(c + i, v[i]);
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (splits > 1 && !ptx::mbar_wait_bounded_cluster(&came, 0, 3 * kWaitNs)) *a.err = (int32_t)kErrWait;

  // ------------------------------------------------------------ finish: 8 features of a token a thread
#pragma unroll 2
  for (int tok = threadIdx.x / kGroups; tok < max(per, 32 / kGroups); tok += kSplitThreads / kGroups) {
    const int row = r0 + rank * per + tok;
    const bool in = tok < per && row >= r_first && row < a.M && c >= f_first && c < a.N;
    float z[8], u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = u[j] = 0.0f;
    if (in) {
      for (int s = 0; s < splits; ++s) {
        const float* p = sums + (s * per + tok) * 128 + group * 8;
        float f[8];
        load8(p, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] += f[j];
        if (GATED) {
          load8(p + 64, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] += f[j];
        }
      }
    }
    if (MODE == FWD) {
      if (in) {
        const float xs = E4M3 ? e.Xs[row] : 1.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          z[j] = E4M3 ? z[j] * ws[0][j] * xs + bs[0][j] : z[j] + bs[0][j];
          if (GATED) u[j] = E4M3 ? u[j] * ws[GATED][j] * xs + bs[GATED][j] : u[j] + bs[GATED][j];
        }
      }
      if (e.Zq) {  // four neighbours share a block
        auto put = [&](const float (&v)[8], int part) {
          float most = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) most = fmaxf(most, finite_abs(v[j]));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
          if (!in) return;
          const uint32_t x = block_exponent(most);
          const float inv = exponent_inverse(x);
          const int64_t line = (int64_t)row * (GATED ? 2 : 1) + part;
          float q[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) q[j] = no_inf(v[j]) * inv;
          *reinterpret_cast<uint2*>(e.Zq + line * a.N + c) =
              make_uint2(pack_e4m3(q[0], q[1], q[2], q[3]), pack_e4m3(q[4], q[5], q[6], q[7]));
          if (c % kBlock == 0) e.Ze[line * ((a.N + kBlock - 1) / kBlock) + c / kBlock] = (uint8_t)x;
        };
        put(z, 0);
        if (GATED) put(u, 1);
      }
      if (GATED) {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = z[j] * sigmoid_fast(z[j]) * u[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = activate(z[j], e.act);
      }
    }
    if (!in) continue;
    if (MODE == DX && e.Xs) {  // the rows of its operand came times the fractions of X's scales
      const float f = 1.0f / scale_fraction(e.Xs[row]);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] *= f;
    }
    const int64_t at = (int64_t)row * a.N + c;
    if (MODE == FWD && e.R) {
      float f[8];
      load8(e.R + at, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] += f[j];
    }
    *reinterpret_cast<uint4*>(e.out + at) = pack8(z);
  }
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, tmem_cols);
  }
}

}  // namespace lin
}  // namespace cusync
