// The products of a linear layer on CTA pairs: one persistent tcgen05 kernel.
//
//   mode   A (M: 256 rows a pair)    B (N: BN columns a pair)       epilogue
//   FWD    X rows                    Wt rows; SwiGLU: BN / 2 gate    scales, bias, checkpoint, activation,
//                                    rows in the first CTA, the up   residual, bf16
//                                    rows N further in the second
//   GRAD   dX: dZ rows               Wt along K                      bf16
//          dWt: dZ along N           X along K (K: tokens)           bf16
//
// "along": the operand is stored with its M (or N) index contiguous rather than the reduction's,
// and the MMA reads it that way through its descriptors; nothing is transposed in memory.  GRAD
// computes both products in one launch, the one with the longer reduction first, whose tail the
// other's tiles fill; dbias's partial sums are added up by a warp that the products leave idle.
//
// What bounds it: under the power cap the MMAs themselves.  4096 x 8192 -> 3584 with SwiGLU in e4m3 took 126 us from
// cool and 146 for seconds (3.82 and 3.30 PFLOP/s), 4096 x 3584 -> 8192 with bias and residual 148 and 153 (1.62 and 1.57),
// both gradients of the former 535 and 590 (1.80 and 1.63), where cuBLAS's bf16 rate is 1.90 in a burst and 1.70
// sustained; the tensor pipe is active in 81 to 91% of cycles.  Small products are bound by 4 us of start and end.
//
// A stage holds 128 bytes x 2 of the reduction for the CTA's 128 rows of A and BN / 2 of B (64 or 48 KB);
// three or four fit beside the epilogue's staging.  Roles, as in the expert layer's products: warp 0 copies A,
// warp kEpi + 2 copies B (TMA, one box each where the widths are multiples of 128 bytes),
// lane 0 of the first CTA's warp 1 issues the MMAs (256 x BN x 32 bytes), the epilogue warps read
// one accumulator of TMEM while the next tile runs into the other.  Tiles are equal, so a
// pair takes tiles t = pair, pair + pairs, ...: row tiles inner within groups of `group`, so that pairs
// at work at the same time share operands in the L2.
//
// Every wait is bounded; an expired one raises the error word and ends the CTA's roles.
#pragma once
#include "lin_math.cuh"
#include "lin_plan.h"
#include "../csrc_moe/moe_ptx.cuh"

namespace cusync {
namespace ptx {

// As umma_bf16 and umma_bf16_pair for e4m3 operands (kind::f8f6f4): 32 k an instruction.
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_e4m3_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor of kind::f8f6f4: fp32 accumulator, e4m3 A and B (type fields 0).
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

}  // namespace ptx

namespace lin {

constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint32_t kErrWait = 3u << 24;  // the pipeline-wait class of the chain kernel's error words

// What both kernels' epilogues of the forward product apply.
struct Epilogue {
  const float *Xs, *Ws;    // E4M3
  const uint16_t *bias, *R;
  uint8_t *Zq, *Ze;
  uint16_t* out;
  int32_t act;
};

// One product: output rows and columns (SwiGLU: of Y), reduction length.
struct GemmShape {
  CUtensorMap mA, mB, mO;
  int32_t M, N, K;
  int32_t m_tiles, n_tiles, group;
  int32_t wideA, wideB;     // one box brings an operand's whole share of a stage
  int32_t along;            // GRAD: A's rows are the reduction's
  int32_t a_rows;           // of a CTA that are copied: 128, or fewer where there are fewer, a multiple of 8
  int32_t b_first;          // B is the first to leave the L2
};
struct GemmArgs {
  GemmShape p[2];           // FWD: [0]
  CUtensorMap mR;           // FWD: the residual, as mO
  Epilogue e;               // FWD; GRAD: Xs, by the fractions of which dX's rows are divided, or NULL
  const float* part;        // GRAD: dbias's partial sums [part_rows][part_cols], or NULL
  uint16_t* sums;
  int32_t part_rows, part_cols;
  int32_t* err;
  int32_t clear;            // this kernel is the call's first: it clears the error word
};

template <int MODE, bool GATED, int BN>
struct GemmCfg {
  // Epilogue warps: four for a tile's 128 rows, two or four such groups side by side over its columns.  Sixteen
  // warps hide each other's latencies (us with eight / sixteen: GeLU, bias and residual, 4096 x 1024 x 4096 38.3 /
  // 35.3, no activation in e4m3 18.5 / 17.2); a gate's registers are too many for that, and the
  // gradients' epilogue is too short (13.6 / 13.8 for 333 x 1000 x 776).
  static constexpr int kEpi = MODE == FWD && !GATED ? 16 : 8;
  static constexpr int kThreads = (kEpi + (MODE == GRAD ? 4 : 3)) * 32;  // GRAD: one for dbias's sums
  static constexpr int kWarpOut = 32 * 1024 / kEpi;        // blocks of 32 rows x 32 columns, 2 KB each
  static constexpr int kBlocks = 2;                        // blocks of 128 bytes of the reduction in a stage
  static constexpr int kABytes = kBlocks * 128 * 128;      // a CTA's share of A in a stage
  static constexpr int kBBytes = kBlocks * BN / 2 * 128;   // and of B
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 192 * 1024 / kStageBytes;
  static constexpr int kSmem = kStages * kStageBytes + kEpi * kWarpOut + 1024;
};

// 16 bytes of bf16 or fp32 values that all lanes read
__device__ __forceinline__ void load8(const uint16_t* p, float (&f)[8]) { unpack8(*reinterpret_cast<const uint4*>(p), f); }
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// What the epilogue of 32 columns needs of them: lane j the scale and bias of column j of each part, which go to
// all lanes by shuffles (read by all lanes 16 bytes at a time a block took longer: 8 against 9.6 us, SwiGLU of 1777 x
// 512 x 1024 in e4m3).  Loaded one block of columns ahead, as a load takes longer than a block.
template <int G>
struct Ahead {
  float ws[G], bs[G];
};
template <bool E4M3, int G>
__device__ __forceinline__ Ahead<G> load_ahead(const Epilogue& e, int N, int c) {
  Ahead<G> v;
  const int col = c + (threadIdx.x & 31);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    v.ws[g] = E4M3 && col < N ? e.Ws[(int64_t)g * N + col] : 0.0f;
    v.bs[g] = e.bias && col < N ? __uint_as_float((uint32_t)e.bias[(int64_t)g * N + col] << 16) : 0.0f;
  }
  return v;
}
// z * scales + bias of 32 columns.  The weights' scale first: that of a row of large values would take z, a sum of
// products of up to 448 each, out of 32 bits before it.
template <bool E4M3>
__device__ __forceinline__ void finish32(const Epilogue& e, float xs, float ws, float bs, float (&z)[32]) {
  if (E4M3) {
#pragma unroll
    for (int j = 0; j < 32; ++j) z[j] = z[j] * __shfl_sync(0xffffffffu, ws, j) * xs;
  }
  if (e.bias) {
#pragma unroll
    for (int j = 0; j < 32; ++j) z[j] += __shfl_sync(0xffffffffu, bs, j);
  }
}

// 32 columns of a row as a block of the checkpoint, `left` of them inside.
__device__ __forceinline__ void store_checkpoint(const Epilogue& e, const float (&z)[32], int left, int64_t row, int part,
                                                 int parts, int N, int c) {
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i < left) most = fmaxf(most, finite_abs(z[i]));
  const uint32_t x = block_exponent(most);
  const float inv = exponent_inverse(x);
  const int64_t line = row * parts + part;
  uint2* q = reinterpret_cast<uint2*>(e.Zq + line * N + c);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (8 * i >= left) break;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = no_inf(z[8 * i + j]) * inv;
    q[i] = make_uint2(pack_e4m3(v[0], v[1], v[2], v[3]), pack_e4m3(v[4], v[5], v[6], v[7]));
  }
  e.Ze[line * ((N + kBlock - 1) / kBlock) + c / kBlock] = (uint8_t)x;
}

// Where a CTA's `span` rows (or columns) of `total` begin that nominally begin at `at`: moved back by a multiple of
// `unit`, so that fewer than `unit` of them lie outside.  The copy engine takes about 8 ns for a row of 128 bytes
// outside of a tensor where it takes 1 for one inside (48 and 128 rows x 384 x 7168 took 11.1 and 12.0 us, 256 rows
// 6.1).  What lies before `at` is another CTA's and not stored here.
__device__ __forceinline__ int span_start(int at, int total, int span, int unit) {
  return min(at, max(0, (total + unit - 1) / unit * unit - span));
}

template <int MODE, bool E4M3, bool GATED, int BN>
__global__ void __launch_bounds__(GemmCfg<MODE, GATED, BN>::kThreads, 1) gemm_kernel(const __grid_constant__ GemmArgs a) {
  using C = GemmCfg<MODE, GATED, BN>;
  constexpr bool kMnB = MODE != FWD;
  constexpr int kStages = C::kStages, kStageBytes = C::kStageBytes, kABytes = C::kABytes, kBBytes = C::kBBytes;
  constexpr int kBlocks = C::kBlocks, kChunk = kBlocks * 64 * 128;  // an "along" operand's 64 columns in a stage
  constexpr int kElems = E4M3 ? 128 : 64;        // reduction elements in 128 bytes
  constexpr int kTileN = GATED ? BN / 2 : BN;    // output columns of a tile
  constexpr int kEpiWarps = C::kEpi, kWarpOut = C::kWarpOut, kOuts = kWarpOut / 2048;
  constexpr int kWarpN = kTileN / (kEpiWarps / 4);  // of an epilogue warp
  constexpr int kBRows = BN / 2;                     // a CTA's share of B
  constexpr int kUnitB = kMnB ? 64 : 32;             // by which B's share may begin elsewhere: chunks, the epilogue's columns
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], drain, came[C::kEpi];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int32_t abort_flag;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)ptx::cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&tfull[i], 1);
      ptx::mbar_init(&tempty[i], kEpiWarps + (rank == 0));  // and the second CTA's warp 1
    }
    for (int i = 0; i < C::kEpi; ++i) ptx::mbar_init(&came[i], 1);
    ptx::mbar_init(&drain, 1);
    ptx::mbar_init_fence();
    abort_flag = 0;
    ptx::prefetch_tmap(&a.p[0].mA);
    ptx::prefetch_tmap(&a.p[0].mB);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(&tmem_slot, 2 * BN);
    ptx::tmem_relinquish_pair();
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::cluster_sync();  // the other CTA's barriers exist
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  if (a.clear && blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;

  const int total0 = a.p[0].m_tiles * a.p[0].n_tiles;
  const int total = total0 + (MODE == GRAD ? a.p[1].m_tiles * a.p[1].n_tiles : 0);
  const int first = blockIdx.x / 2, step = gridDim.x / 2;
  // tile t's product, and its place: groups of `group` row tiles, columns outer, rows inner
  auto tile = [&](int t, int& m0, int& n0) -> const GemmShape& {
    const bool second = MODE == GRAD && t >= total0;
    const GemmShape& p = a.p[second ? 1 : 0];
    if (second) t -= total0;
    const int per = p.group * p.n_tiles, g = t / per, r = t - g * per;
    const int rows = min(p.group, p.m_tiles - g * p.group);
    const int n = r / rows;
    m0 = (g * p.group + r - n * rows) * 256;
    n0 = n * kTileN;
    return p;
  };

  if (warp == 0 || warp == kEpiWarps + 2) {
    // ------------------------------------------------------------ copies
    const bool copies_a = warp == 0;
    const bool leaves = MODE == FWD && !copies_a && a.p[0].b_first;
    const uint64_t pol = leaves ? ptx::l2_policy_evict_first() : ptx::l2_policy_evict_normal();
    const bool one = ptx::elect_one();
    uint8_t* base = ring + (copies_a ? 0 : kABytes);
    const uint32_t full0 = ptx::mapa(&full[0], 0);
    uint32_t it = 0, st = 0, par = 1;
    bool ok = true;
    for (int t = first; t < total && ok && !abort_flag; t += step) {
      int m0, n0;
      const GemmShape& p = tile(t, m0, n0);
      const int nkb = (p.K + kElems - 1) / kElems;  // blocks of 128 bytes
      const bool mn = MODE == GRAD && (!copies_a || p.along), wide = copies_a ? p.wideA : p.wideB;
      const CUtensorMap* map = copies_a ? &p.mA : &p.mB;
      // this CTA's first row (or column) of the operand
      const int r0 = copies_a ? span_start(m0 + 128 * rank, p.M, 128, mn ? 64 : 32)
                     : GATED  ? span_start(n0, p.N, kBRows, kUnitB) + rank * p.N
                              : span_start(n0 + kBRows * rank, p.N, kBRows, kUnitB);
      const int block = (copies_a ? p.a_rows : kBRows) * 128;  // bytes of a block
      const uint32_t a_bytes = 2 * p.a_rows * 128;
      // the second CTA's share, where none of it is inside, is not copied: what stands there counts for outputs that no
      // one stores
      const int both_a = m0 + 128 < p.M ? 2 : 1, both_b = GATED || n0 + kBRows < p.N ? 2 : 1;
      const bool skip = rank == 1 && (copies_a ? both_a : both_b) == 1;
      for (int kb = 0; kb < nkb; kb += kBlocks, ++it) {
        ok = ptx::mbar_wait_bounded(&empty[st], par, kWaitNs);
        if (!ok) break;
        const uint32_t bar = full0 + 8 * st;  // both CTAs' copies complete on the first one's barrier
        uint8_t* dst = base + st * kStageBytes;
        const bool half = kb + 1 == nkb;  // the second block holds nothing
        if (one) {
          if (copies_a && rank == 0) {
            // an operand's second block is counted where a box brings it, even from outside
            const uint32_t as = (MODE == GRAD && p.along) || p.wideA || !half ? a_bytes : a_bytes / 2;
            const uint32_t bs = kMnB || p.wideB || !half ? kBBytes : kBBytes / 2;
            ptx::mbar_arrive_expect_tx(&full[st], both_a * as + both_b * bs);
          }
          if (skip) {
          } else if (mn) {  // chunks of 64 columns x 128 k
            if (wide) {
              ptx::tma_load_3d_to_leader(dst, map, bar, 0, kb * 64, r0 / 64, pol);
            } else {
              ptx::tma_load_2d_to_leader(dst, map, bar, r0, kb * 64, pol);
              if (copies_a || kBRows > 64) ptx::tma_load_2d_to_leader(dst + kChunk, map, bar, r0 + 64, kb * 64, pol);
            }
          } else {   // blocks of 128 bytes
            if (wide) {
              ptx::tma_load_3d_to_leader(dst, map, bar, 0, r0, kb, pol);
            } else {
              ptx::tma_load_2d_to_leader(dst, map, bar, kb * kElems, r0, pol);
              if (!half) ptx::tma_load_2d_to_leader(dst + block, map, bar, (kb + 1) * kElems, r0, pol);
            }
          }
        }
        __syncwarp();
        if (++st == kStages) {
          st = 0;
          par ^= 1;
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (!ok && lane == 0) {
      abort_flag = 1;
      *a.err = (int32_t)kErrWait;
    }
    __syncwarp();
    // after an abort: wait, bounded, for the copies still in flight (all complete on the first CTA's `full`)
    if (abort_flag && copies_a && lane == 0 && rank == 0)
      for (uint32_t i = it > (uint32_t)kStages ? it - kStages : 0; i < it; ++i)
        ptx::mbar_wait_bounded(&full[i % kStages], (i / kStages) & 1, kWaitNs);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    bool ok = true;
    if (rank == 0) {
      const uint32_t ring0 = __shfl_sync(0xffffffffu, ptx::smem_u32(ring), 0);
      const bool one = ptx::elect_one();  // the lane whose MMAs its commits cover
      constexpr uint32_t kIdesc = (E4M3 ? ptx::idesc_e4m3_f32(256, BN) : ptx::idesc_bf16_f32(256, BN)) |
                                  (kMnB ? ptx::kIdescBMn : 0);
      uint32_t st = 0, par = 0, acc = 0;
      for (int t = first; t < total && ok && !abort_flag; t += step, ++acc) {
        const uint32_t buf = acc & 1, use = acc >> 1;
        int m0, n0;
        const GemmShape& p = tile(t, m0, n0);
        const int nkb = (p.K + kElems - 1) / kElems;
        const bool along = MODE == GRAD && p.along;
        const int a_block = p.a_rows * 128;
        const uint32_t idesc = kIdesc | (along ? ptx::kIdescAMn : 0);
        ok = ptx::mbar_wait_bounded_cluster(&tempty[buf], (use & 1) ^ 1, kWaitNs) && !abort_flag;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem + buf * BN;
        for (int kb = 0; kb < nkb; kb += kBlocks) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(&full[st], par, kWaitNs));
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t sA = ring0 + st * kStageBytes, sB = sA + kABytes;
          const uint64_t dA = along ? ptx::smem_desc_mn128(sA, kChunk) : ptx::smem_desc_k128(sA);
          const uint64_t dB = kMnB ? ptx::smem_desc_mn128(sB, kChunk) : ptx::smem_desc_k128(sB);
          // 32 bytes of the reduction at a time; the last stage's steps that hold none of it are left out
          const int steps = (p.K - kb * kElems + kElems / 4 - 1) / (kElems / 4);
#pragma unroll
          for (int s = 0; s < 4 * kBlocks; ++s) {
            if (s >= steps) break;
            if (!one) continue;
            // along the reduction: 32 bytes of a block's rows; across it: 16 rows of 128 bytes
            const uint64_t mn = (uint64_t)(s * 2048) >> 4;
            const uint64_t oA = along ? mn : (uint64_t)(s / 4 * a_block + s % 4 * 32) >> 4;
            const uint64_t oB = kMnB ? mn : (uint64_t)(s / 4 * (kBBytes / kBlocks) + s % 4 * 32) >> 4;
            if (E4M3) ptx::umma_e4m3_pair(d, dA + oA, dB + oB, idesc, kb || s);
            else ptx::umma_bf16_pair(d, dA + oA, dB + oB, idesc, kb || s);
          }
          if (one) ptx::umma_commit_pair_multicast(&empty[st], 0x3);
          __syncwarp();
          if (++st == kStages) {
            st = 0;
            par ^= 1;
          }
        }
        if (!ok) break;
        if (one) ptx::umma_commit_pair_multicast(&tfull[buf], 0x3);
        __syncwarp();
      }
      if (!ok || abort_flag) {
        abort_flag = 1;
        *a.err = (int32_t)kErrWait;
        if (one) ptx::umma_commit_pair_multicast(&drain, 0x3);  // MMAs still in flight
        ptx::mbar_wait_bounded(&drain, 0, kWaitNs);
      }
    } else {
      // the second CTA's: accumulators back to the first as the epilogue here is done with them (a
      // release across the pair waits for the thread's own stores, and this warp has none)
      uint32_t acc = 0;
      for (int t = first; t < total && !abort_flag; t += step, ++acc) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(&tempty[acc & 1], (acc >> 1) & 1, kWaitNs));
        if (!ok) break;
        if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa(&tempty[acc & 1], 0));
        __syncwarp();
      }
      if (!ok) {
        abort_flag = 1;
        *a.err = (int32_t)kErrWait;
      }
    }
    __syncwarp();
  } else if (warp < kEpiWarps + 2) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    uint8_t* stage = ring + kStages * kStageBytes + (warp - 2) * kWarpOut;
    const Epilogue& e = a.e;
    uint32_t acc = 0, blocks = 0, loads = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += step, ++acc) {
      int m0, n0;
      const GemmShape& p = tile(t, m0, n0);
      const uint32_t buf = acc & 1, use = acc >> 1;
      const int row0 = span_start(m0 + 128 * rank, p.M, 128, MODE == GRAD && p.along ? 64 : 32) + 32 * quarter, row = row0 + lane;
      const bool rows = row0 >= m0 + 128 * rank && row0 < p.M;  // of this CTA's own
      const bool in = rows && row < p.M;
      // this warp's first output column, and the first of its blocks of 32 from there on that is the tile's own
      const int own = GATED ? n0 : n0 + half * kWarpN / kBRows * kBRows;  // of the share of B that they come from
      const int c0 = span_start(own, p.N, kBRows, kUnitB) + (GATED ? half * kWarpN : half * kWarpN % kBRows);
      const int i0 = rows ? max(0, own - c0) / 32 : kWarpN / 32;
      float xs = 1.0f;
      if (E4M3 && in) xs = e.Xs[row];
      const bool divide = MODE == GRAD && e.Xs && !p.along;
      if (divide && in) xs = 1.0f / scale_fraction(e.Xs[row]);
      constexpr int G = GATED ? 2 : 1;
      Ahead<G> now;
      if (MODE == FWD) now = load_ahead<E4M3, G>(e, p.N, c0 + 32 * i0);
      ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleepy(&tfull[buf], use & 1, kWaitNs) && !abort_flag);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t d = tmem + buf * BN + lanes;
#pragma unroll 1
      for (int i = i0; i < kWarpN / 32; ++i) {
        const int at = half * kWarpN + 32 * i, c = c0 + 32 * i, left = p.N - c;  // columns from c on
        if (left <= 0) break;
        // this block of the staging, free once the store before the last (the last, with one block) has read it; the
        // residual's 32 x 32 come into it first
        uint8_t* block = stage + (blocks % kOuts) * 2048;
        if (lane == 0) {
          ptx::bulk_wait_group_read<kOuts - 1>();
          if (MODE == FWD && e.R) {
            ptx::mbar_arrive_expect_tx(&came[warp - 2], 2048);
            ptx::tma_load_2d(block, &a.mR, &came[warp - 2], c, row0, ptx::l2_policy_evict_first());
          }
        }
        __syncwarp();
        float z[32], u[32];
        {
          uint32_t v[32];
          ptx::tmem_ld_32x32b_x32(d + at, v);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(v[j]);
        }
        if (GATED) {
          uint32_t v[32];
          ptx::tmem_ld_32x32b_x32(d + BN / 2 + at, v);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) u[j] = __uint_as_float(v[j]);
        }
        if (MODE == FWD) {
          finish32<E4M3>(e, xs, now.ws[0], now.bs[0], z);
          if (GATED) finish32<E4M3>(e, xs, now.ws[G - 1], now.bs[G - 1], u);
          if (e.Zq && in) {
            store_checkpoint(e, z, left, row, 0, GATED ? 2 : 1, p.N, c);
            if (GATED) store_checkpoint(e, u, left, row, 1, 2, p.N, c);
          }
          if (GATED) {
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = z[j] * sigmoid_fast(z[j]) * u[j];
          } else if (e.act != ACT_NONE) {
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = activate(z[j], e.act);
          }
          if (i + 1 < kWarpN / 32) now = load_ahead<E4M3, G>(e, p.N, c + 32);
        }
        if (divide) {
#pragma unroll
          for (int j = 0; j < 32; ++j) z[j] *= xs;
        }
        // a lane's 32 columns: four 16-byte pieces of 64-byte rows, placed as the maps' 64-byte swizzle
        // has them; rows and columns outside the matrix are not written
        if (MODE == FWD && e.R) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(&came[warp - 2], loads & 1, kWaitNs));
          ++loads;
          if (!ok) break;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4* piece = reinterpret_cast<uint4*>(block + lane * 64 + ((j ^ (lane / 2)) & 3) * 16);
          if (MODE == FWD && e.R) {
            float f[8];
            unpack8(*piece, f);
#pragma unroll
            for (int k = 0; k < 8; ++k) z[8 * j + k] += f[k];
          }
          uint32_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = pack2(z[8 * j + 2 * k], z[8 * j + 2 * k + 1]);
          *piece = make_uint4(v[0], v[1], v[2], v[3]);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::tma_store_2d(&p.mO, block, c, row0);
          ptx::bulk_commit_group();
        }
        ++blocks;
      }
      if (!ok) break;
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&tempty[buf]);
    }
    if (lane == 0) ptx::bulk_wait_group_read<0>();  // the stores still read this warp's blocks
    if (!ok && lane == 0) {
      abort_flag = 1;
      *a.err = (int32_t)kErrWait;
    }
    __syncwarp();
  } else if (MODE == GRAD && a.part) {
    // ------------------------------------------------------------ dbias: 32 columns at a time, rows in order
    for (int c = blockIdx.x * 32 + lane; c < a.part_cols; c += gridDim.x * 32) {
      float sum = 0.0f;
      for (int r = 0; r < a.part_rows; r += 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = r + k < a.part_rows ? a.part[(int64_t)(r + k) * a.part_cols + c] : 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += v[k];
      }
      a.sums[c] = __bfloat16_as_ushort(__float2bfloat16_rn(sum));
    }
    __syncwarp();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // both CTAs are done with the pair's TMEM and barriers
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 2 * BN);
  }
}

}  // namespace lin
}  // namespace cusync
