// The products of an expert layer: one persistent tcgen05 kernel per product.
//
// A tile is 128 rows of one expert (the plan aligns an expert's rows to 128) x BN columns,
// or, for a weight gradient, 128 x BN of one expert's matrix.  With PAIR = 2 a pair of CTAs
// (cta_group::2) computes 256 rows: each holds its 128 rows of A and half of B's columns,
// so that a 128 x 256 x 64 block costs an SM 32 KB of loads, not 48 KB.  One CTA per SM
// walks its tiles with a fixed stride:
//   warp 0     copies: TMA boxes of the weights and of the slot-ordered rows.
//   warp 1     TMEM owner; lane 0 (of a pair's first CTA) issues tcgen05.mma (fp32
//              accumulators).
//   warps 2-9  epilogue: two warps per TMEM lane quarter, a thread per row.
// Accumulators are double-buffered where two fit in TMEM's 512 columns.
//
//   mode   rows x columns          A            B                       epilogue
//   FWD1   slots x N1              X by slot    W1t[e]                  h = act(z), bf16
//   FWD1G  the same                X (gather)
//   FWD2   slots x D               H            W2t[e]                  O, fp32
//   BWD1   slots x N1              X, dY        W1t[e]; W2t[e] along N  z and dH = dY W2 side by
//                                                                       side: dZ and w h (bf16),
//                                                                       partial sums of dH h
//   DX     slots x D               dZ           W1t[e] along N          dX per slot, fp32
//   DW1    G*N1 x D (per expert)   dZ along M   X along N               bf16
//   DW2    D x N1 (per expert)     dY along M   w H along N             bf16
//
// "along M/N": the operand is stored with that index contiguous rather than K, and the MMA
// reads it that way (instruction and shared-memory descriptors), so no operand is ever
// transposed in memory.
//
// X by slot: a copy in slot order (dispatch_kernel).  The gather (tile::gather4, four rows a
// copy through the plan's row indices) needs no such copy, but brings 128 rows x 64 columns
// in 1.25 us, three times what the MMAs of a 128 x 256 x 64 block take (first product of
// 4096 tokens x 8 of 64 experts, D = 2048, N1 = 1024: 609 us): it is for tiles of few rows.
//
// A row behind an expert's last one gets no store in the forward pass; its accumulator
// rows hold whatever the ring held, and rows do not mix.  In the weight gradients K runs
// over slots: there dispatch_kernel and BWD1 stored zeros for such rows.
//
// Every wait is bounded; an expired one raises the error word and ends the CTA's roles.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "moe_plan.cuh"
#include "ptx.cuh"

namespace cusync {
namespace moe {

enum : int { FWD1 = 0, FWD2 = 1, BWD1 = 2, DX = 3, DW1 = 4, DW2 = 5, FWD1G = 6 };

constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kGemmThreads = 320;
constexpr uint32_t kErrWait = 3u << 24;  // the pipeline-wait class of the chain kernel's error words

struct GemmArgs {
  CUtensorMap mA;    // X, H, dZ or dY
  CUtensorMap mA2;   // BWD1: dY
  CUtensorMap mB;    // W1t, W2t, X or w H
  CUtensorMap mB2;   // BWD1: W2t
  int32_t* plan;
  const float* weights;
  void* out;         // H, O, dZ, dX per slot, dW1t or dW2t
  void* out2;        // BWD1: w H
  float* part;       // BWD1: partial sums of dH h, [slot][2 * column tiles]
  int64_t counts, offsets, tiles, row_of;  // plan words; tiles: of the launch's 128 or 256 rows
  int32_t T, k, E;
  int32_t M;         // DW: rows of an expert's matrix
  int32_t N;         // output columns (FWD1, BWD1: N1)
  int32_t K;         // reduction length (DW: the expert's rows)
  int32_t col_tiles, m_tiles;
};

template <int MODE, int ACT, int BN, int PAIR>
struct GemmCfg {
  static constexpr bool kDw = MODE == DW1 || MODE == DW2;
  static constexpr bool kBwd1 = MODE == BWD1;
  static constexpr bool kFwd1 = MODE == FWD1 || MODE == FWD1G;
  static constexpr bool kGather = MODE == FWD1G;
  static constexpr bool kPairB = ACT == 1 && (kFwd1 || kBwd1);  // gate and up columns in one tile
  static constexpr bool kMnA = kDw;
  static constexpr bool kMnB = kDw || MODE == DX;
  static constexpr int kOutCols = kPairB ? BN / 2 : BN;  // output columns of a tile
  static constexpr int kABytes = 128 * 128;
  static constexpr int kBBytes = BN / PAIR * 128;
  static constexpr int kD2 = kBwd1 ? kOutCols : 0;       // columns of BWD1's second accumulator
  static constexpr int kStageBytes = kABytes + kBBytes + (kBwd1 ? kABytes + kD2 / PAIR * 128 : 0);
  static constexpr int kRing = 192 * 1024;
  static constexpr int kStageOut = 8 * 4096;              // epilogue: 32 rows of 128 bytes for each warp
  static constexpr int kStages = kRing / kStageBytes < 8 ? kRing / kStageBytes : 8;
  static constexpr int kAccCols = BN + kD2;
  static constexpr int kAccs = 2 * kAccCols <= 512 ? 2 : 1;
  static constexpr int kTmemCols = kAccs * kAccCols <= 128 ? 128 : kAccs * kAccCols <= 256 ? 256 : 512;
  static constexpr int kSmemBytes = kStages * kStageBytes + kStageOut + 1024;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// 1 / (1 + e^-x); the fast exponential and division are within a few 1e-7 of it
__device__ __forceinline__ float sigmoid_fast(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
// The factor of z in GeLU_tanh(z) = z sigmoid(2 c (z + 0.044715 z^3))
__device__ __forceinline__ float gelu_gate(float z) {
  return sigmoid_fast(2.0f * kGeluC * (z + 0.044715f * z * z * z));
}

// One tile of a launch.
struct Tile {
  int32_t e, slot0, rows, m0, n0, nkb;
};

template <int MODE, int ACT, int BN, int PAIR>
__device__ __forceinline__ int32_t tile_total(const GemmArgs& a) {
  if (GemmCfg<MODE, ACT, BN, PAIR>::kDw) return a.E * a.m_tiles * a.col_tiles;
  return a.plan[PAIR == 2 ? PLAN_PAIRS : PLAN_TILES] * a.col_tiles;
}

template <int MODE, int ACT, int BN, int PAIR>
__device__ __forceinline__ Tile tile_at(const GemmArgs& a, int32_t t) {
  using C = GemmCfg<MODE, ACT, BN, PAIR>;
  Tile r;
  if (C::kDw) {
    const int32_t per = a.m_tiles * a.col_tiles;
    r.e = t / per;
    const int32_t q = t - r.e * per;
    r.m0 = (q % a.m_tiles) * (128 * PAIR);
    r.n0 = (q / a.m_tiles) * BN;
    r.slot0 = a.plan[a.offsets + r.e];
    r.rows = a.plan[a.counts + r.e];
    r.nkb = (r.rows + 63) / 64;
  } else {
    const int32_t rt = t / a.col_tiles;
    const int4 er = *reinterpret_cast<const int4*>(a.plan + a.tiles + 4 * rt);
    r.e = er.x;
    r.slot0 = er.y;
    r.rows = er.z;
    r.m0 = 0;
    r.n0 = (t - rt * a.col_tiles) * C::kOutCols;
    r.nkb = (a.K + 63) / 64;
  }
  return r;
}

// A CTA's tiles, read one ahead: the plan's entry of a tile is a trip to L2 that no role
// should wait for between two tiles.
template <int MODE, int ACT, int BN, int PAIR>
struct Walk {
  const GemmArgs& a;
  const int32_t total;
  int32_t t;
  Tile next;
  __device__ __forceinline__ Walk(const GemmArgs& args, int32_t n) : a(args), total(n), t(blockIdx.x / PAIR) {
    if (t < total) next = tile_at<MODE, ACT, BN, PAIR>(a, t);
  }
  __device__ __forceinline__ bool take(Tile& q) {
    if (t >= total) return false;
    q = next;
    t += gridDim.x / PAIR;
    if (t < total) next = tile_at<MODE, ACT, BN, PAIR>(a, t);
    return true;
  }
};

// 32 rows x 128 bytes, staged in shared memory (16-byte pieces, swizzled so that neither
// side conflicts) and stored as whole 128-byte rows, four to an instruction.  `mine` is this
// lane's row; row r of the warp goes to out + r * pitch when r < rows, its 16-byte pieces
// below `pieces`.
template <int PIECES>
__device__ __forceinline__ void store_rows(uint8_t* stage, const uint32_t (&mine)[4 * PIECES], uint8_t* out,
                                           int64_t pitch, int rows, int pieces, int lane) {
  constexpr int kRowsEach = 32 / PIECES;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
    *reinterpret_cast<uint4*>(stage + lane * (16 * PIECES) + ((i ^ (lane * PIECES / 8)) & (PIECES - 1)) * 16) =
        make_uint4(mine[4 * i], mine[4 * i + 1], mine[4 * i + 2], mine[4 * i + 3]);
  __syncwarp();
  const int piece = lane % PIECES;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int r = i * kRowsEach + lane / PIECES;
    const uint4 v = *reinterpret_cast<const uint4*>(stage + r * (16 * PIECES) +
                                                    ((piece ^ (r * PIECES / 8)) & (PIECES - 1)) * 16);
    if (r < rows && piece < pieces) *reinterpret_cast<uint4*>(out + r * pitch + piece * 16) = v;
  }
}

template <int MODE, int ACT, int BN, int PAIR>
__global__ void __launch_bounds__(kGemmThreads, 1) moe_gemm_kernel(const __grid_constant__ GemmArgs a) {
  using C = GemmCfg<MODE, ACT, BN, PAIR>;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t full[C::kStages], empty[C::kStages], tfull[2], tempty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int32_t abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR == 2 ? (int)ptx::cluster_ctarank() : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&tfull[i], 1);
      ptx::mbar_init(&tempty[i], 8 * PAIR);
    }
    ptx::mbar_init(&drain, 1);
    ptx::mbar_init_fence();
    abort_flag = 0;
    ptx::prefetch_tmap(&a.mA);
    ptx::prefetch_tmap(&a.mB);
    if (C::kBwd1) {
      ptx::prefetch_tmap(&a.mA2);
      ptx::prefetch_tmap(&a.mB2);
    }
  }
  if (warp == 1) {
    if (PAIR == 2) {
      ptx::tmem_alloc_pair(&tmem_slot, C::kTmemCols);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(&tmem_slot, C::kTmemCols);
      ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
  }
  __syncthreads();
  if (PAIR == 2) ptx::cluster_sync();  // the other CTA's barriers exist
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  Walk<MODE, ACT, BN, PAIR> walk(a, tile_total<MODE, ACT, BN, PAIR>(a));
  Tile q;

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    const uint64_t keep = ptx::l2_policy_evict_last(), stream = ptx::l2_policy_evict_normal();
    uint32_t it = 0, st = 0, par = 1;
    const uint32_t full0 = PAIR == 2 ? ptx::mapa(&full[0], 0) : 0;
    while (!abort_flag && walk.take(q)) {
      // a lane's four gathered rows, as token indices; -1 (a slot behind the last row)
      // becomes T, outside the tensor, read as zero
      int4 tok = make_int4(a.T, a.T, a.T, a.T);
      if (C::kGather && 4 * lane < q.rows) {
        const int4 r = *reinterpret_cast<const int4*>(a.plan + a.row_of + q.slot0 + 4 * lane);
        auto token = [&](int32_t x) { return x < 0 ? a.T : x / a.k; };
        tok = make_int4(token(r.x), token(r.y), token(r.z), token(r.w));
      }
      const int live = (q.rows + 3) / 4;           // lanes whose rows a gathered tile needs
      // this CTA's rows and columns of the tile
      const int32_t slot = q.slot0 + (C::kDw ? 0 : 128 * rank), m0 = q.m0 + 128 * rank;
      const int boxes = C::kDw ? 0 : (q.rows - 128 * rank + 31) / 32;  // 32-row boxes of A
      const int32_t nb = q.n0 + (C::kPairB ? 0 : rank * (BN / 2)), n2 = q.n0 + rank * (C::kD2 / 2);
      uint32_t bytes = PAIR * (C::kBBytes + (C::kBwd1 ? C::kD2 / PAIR * 128 : 0));
      if (C::kGather) bytes += live * 512;
      else if (C::kDw) bytes += PAIR * C::kABytes;
      else if (PAIR == 2 || C::kBwd1) bytes += (C::kBwd1 ? 2 : 1) * (q.rows > 128 ? 2 : 1) * C::kABytes;
      else bytes += boxes * 4096;
      bool ok = true;
      // Every lane waits for the slot and issues its own copies: nothing orders the lanes,
      // since the barrier's phase cannot end before lane 0's arrival.
      for (int kb = 0; kb < q.nkb; ++kb, ++it) {
        ok = ptx::mbar_wait_bounded(&empty[st], par, kWaitNs);
        if (!ok) break;
        uint8_t* sA = ring + st * C::kStageBytes;
        uint8_t* sB = sA + C::kABytes;
        uint8_t* sA2 = sB + C::kBBytes;
        uint8_t* sB2 = sA2 + C::kABytes;
        uint64_t* bar = &full[st];
        // in a pair both CTAs' copies complete on the first one's barrier
        const uint32_t bar0 = full0 + 8 * st;
        auto load2 = [&](void* dst, const CUtensorMap* m, int32_t c0, int32_t c1, uint64_t pol) {
          if (PAIR == 2) ptx::tma_load_2d_to_leader(dst, m, bar0, c0, c1, pol);
          else ptx::tma_load_2d(dst, m, bar, c0, c1, pol);
        };
        auto load3 = [&](void* dst, const CUtensorMap* m, int32_t c0, int32_t c1, int32_t c2, uint64_t pol) {
          if (PAIR == 2) ptx::tma_load_3d_to_leader(dst, m, bar0, c0, c1, c2, pol);
          else ptx::tma_load_3d(dst, m, bar, c0, c1, c2, pol);
        };
        if (lane == 0 && rank == 0) ptx::mbar_arrive_expect_tx(bar, bytes);
        if (++st == C::kStages) {
          st = 0;
          par ^= 1;
        }
        const int32_t kc = kb * 64;
        // A
        if (C::kGather) {
          if (lane < live) ptx::tma_gather4(sA + lane * 512, &a.mA, bar, kc, tok, keep);
        } else if (C::kDw) {
          if (lane < 2) load2(sA + lane * 8192, &a.mA, m0 + 64 * lane, slot + kc, keep);
        } else if (PAIR == 2 || C::kBwd1) {
          if (lane == 1 && boxes > 0) load2(sA, &a.mA, kc, slot, keep);
          if (C::kBwd1 && lane == 2 && boxes > 0) load2(sA2, &a.mA2, kc, slot, keep);
        } else {
          if (lane < boxes) load2(sA + lane * 4096, &a.mA, kc, slot + 32 * lane, keep);
        }
        // B: this CTA's columns
        if (C::kDw) {
          if (lane < BN / PAIR / 64) load2(sB + lane * 8192, &a.mB, nb + 64 * lane, slot + kc, keep);
        } else if (MODE == DX) {
          if (lane < BN / PAIR / 64) load3(sB + lane * 8192, &a.mB, nb + 64 * lane, kc, q.e, stream);
        } else if (lane == 0) {
          if (!C::kPairB) {
            load3(sB, &a.mB, kc, nb, q.e, stream);
          } else if (PAIR == 2) {
            load3(sB, &a.mB, kc, nb, 2 * q.e + rank, stream);  // gate columns; up columns
          } else {
            load3(sB, &a.mB, kc, nb, 2 * q.e, stream);
            load3(sB + C::kBBytes / 2, &a.mB, kc, nb, 2 * q.e + 1, stream);
          }
        }
        if (C::kBwd1 && lane < C::kD2 / PAIR / 64) load3(sB2 + lane * 8192, &a.mB2, n2 + 64 * lane, kc, q.e, stream);
      }
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) {
          abort_flag = 1;
          a.plan[PLAN_ERR] = (int32_t)kErrWait;
        }
        break;
      }
    }
    __syncwarp();
    // after an abort: wait, bounded, for the copies still in flight
    if (abort_flag && lane == 0 && rank == 0)
      for (uint32_t i = it > (uint32_t)C::kStages ? it - C::kStages : 0; i < it; ++i)
        ptx::mbar_wait_bounded(&full[i % C::kStages], (i / C::kStages) & 1, kWaitNs);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (lane == 0 && rank == 0) {
      constexpr uint32_t majors = (C::kMnA ? ptx::kIdescAMn : 0) | (C::kMnB ? ptx::kIdescBMn : 0);
      constexpr uint32_t idesc = ptx::idesc_bf16_f32(128 * PAIR, BN) | majors;
      constexpr uint32_t idesc2 = ptx::idesc_bf16_f32(128 * PAIR, C::kBwd1 ? C::kD2 : BN) | ptx::kIdescBMn;
      auto mma = [&](uint32_t d, uint64_t da, uint64_t db, uint32_t id, uint32_t more) {
        if (PAIR == 2) ptx::umma_bf16_pair(d, da, db, id, more);
        else ptx::umma_bf16(d, da, db, id, more);
      };
      auto commit = [&](uint64_t* bar) {
        if (PAIR == 2) ptx::umma_commit_pair_multicast(bar, 0x3);
        else ptx::umma_commit(bar);
      };
      uint32_t st = 0, par = 0, acc = 0;
      bool ok = true;
      while (ok && !abort_flag && walk.take(q)) {
        if (q.nkb == 0) continue;  // an expert without rows: the epilogue writes zeros
        const uint32_t buf = acc % C::kAccs, use = acc / C::kAccs;
        ++acc;
        ok = (PAIR == 2 ? ptx::mbar_wait_bounded_cluster(&tempty[buf], (use & 1) ^ 1, kWaitNs)
                        : ptx::mbar_wait_bounded(&tempty[buf], (use & 1) ^ 1, kWaitNs)) &&
             !abort_flag;
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem + buf * C::kAccCols;
        for (int kb = 0; kb < q.nkb; ++kb) {
          ok = ptx::mbar_wait_bounded(&full[st], par, kWaitNs);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t sA = ptx::smem_u32(ring + st * C::kStageBytes);
          const uint32_t sB = sA + C::kABytes, sA2 = sB + C::kBBytes, sB2 = sA2 + C::kABytes;
          // 16 k: 32 bytes of a K-contiguous row, or 16 rows of 128 bytes
          constexpr uint64_t stepA = C::kMnA ? 2048 >> 4 : 32 >> 4, stepB = C::kMnB ? 2048 >> 4 : 32 >> 4;
          const uint64_t dA = C::kMnA ? ptx::smem_desc_mn128(sA) : ptx::smem_desc_k128(sA);
          const uint64_t dB = C::kMnB ? ptx::smem_desc_mn128(sB) : ptx::smem_desc_k128(sB);
#pragma unroll
          for (int s = 0; s < 4; ++s) mma(d, dA + s * stepA, dB + s * stepB, idesc, kb || s);
          if (C::kBwd1) {
            const uint64_t dA2 = ptx::smem_desc_k128(sA2), dB2 = ptx::smem_desc_mn128(sB2);
#pragma unroll
            for (int s = 0; s < 4; ++s)
              mma(d + BN, dA2 + s * (32 >> 4), dB2 + s * (2048 >> 4), idesc2, kb || s);
          }
          commit(&empty[st]);
          if (++st == C::kStages) {
            st = 0;
            par ^= 1;
          }
        }
        if (!ok) break;
        commit(&tfull[buf]);
      }
      if (!ok || abort_flag) {
        abort_flag = 1;
        a.plan[PLAN_ERR] = (int32_t)kErrWait;
        commit(&drain);  // MMAs still in flight
        ptx::mbar_wait_bounded(&drain, 0, kWaitNs);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = (warp - 2) >> 2;  // TMEM lane quarter; every other 32 columns
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    uint8_t* stage = ring + C::kStages * C::kStageBytes + (warp - 2) * 4096;
    const int row0 = quarter * 32;
    uint32_t acc = 0;
    while (walk.take(q)) {
      const bool empty_tile = q.nkb == 0;
      const uint32_t buf = acc % C::kAccs, use = acc / C::kAccs;
      if (!empty_tile) {
        ++acc;
        const bool ok = ptx::mbar_wait_sleepy(&tfull[buf], use & 1, kWaitNs) && !abort_flag;
        if (!__all_sync(0xffffffffu, ok)) {
          abort_flag = 1;
          if (lane == 0) a.plan[PLAN_ERR] = (int32_t)kErrWait;
          break;
        }
        ptx::tc_fence_after();
      }
      const uint32_t d = tmem + buf * C::kAccCols + lanes;
      // this warp's 32 rows: of the matrix (weight gradients) or of the slots, `rows` of them real
      const int r0 = 128 * rank + row0, rows = q.rows - r0;
      const int64_t slot0 = (int64_t)q.slot0 + r0, slot = slot0 + lane;
      const bool live = lane < rows;
      if (C::kFwd1) {
#pragma unroll 1
        for (int c = half * 32; c < C::kOutCols; c += 64) {
          uint32_t z[32], u[32], p[16];
          ptx::tmem_ld_32x32b_x32(d + c, z);
          if (C::kPairB) ptx::tmem_ld_32x32b_x32(d + C::kOutCols + c, u);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float h[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const float x = __uint_as_float(z[2 * i + b]);
              h[b] = C::kPairB ? x * sigmoid_fast(x) * __uint_as_float(u[2 * i + b]) : x * gelu_gate(x);
            }
            p[i] = pack2(h[0], h[1]);
          }
          const int n = q.n0 + c;
          store_rows<4>(stage, p, reinterpret_cast<uint8_t*>(a.out) + (slot0 * a.N + n) * 2, (int64_t)a.N * 2,
                        rows, (a.N - n) / 8, lane);
        }
      } else if (MODE == FWD2 || MODE == DX) {
#pragma unroll 1
        for (int c = half * 32; c < BN; c += 64) {
          uint32_t z[32];
          ptx::tmem_ld_32x32b_x32(d + c, z);
          ptx::tmem_ld_wait();
          const int n = q.n0 + c;
          store_rows<8>(stage, z, reinterpret_cast<uint8_t*>(a.out) + (slot0 * a.N + n) * 4, (int64_t)a.N * 4,
                        rows, (a.N - n) / 4, lane);
        }
      } else if (MODE == BWD1) {
        float w = 0.0f, dot = 0.0f;
        if (live) {
          const int r = a.plan[a.row_of + slot];
          w = r >= 0 ? a.weights[r] : 0.0f;
        }
        constexpr int G = C::kPairB ? 2 : 1;
        const int64_t pitch = (int64_t)G * a.N * 2;
#pragma unroll 1
        for (int c = half * 32; c < C::kOutCols; c += 64) {
          const int n = q.n0 + c;
          uint32_t pz[16], pu[16], ph[16];
#pragma unroll
          for (int i0 = 0; i0 < 32; i0 += 16) {
            uint32_t z[16], u[16], g[16];
            ptx::tmem_ld_32x32b_x16(d + c + i0, z);
            if (C::kPairB) ptx::tmem_ld_32x32b_x16(d + C::kOutCols + c + i0, u);
            ptx::tmem_ld_32x32b_x16(d + BN + c + i0, g);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float vz[2], vu[2], vh[2];
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const float zz = __uint_as_float(z[2 * j + b]), dh = __uint_as_float(g[2 * j + b]);
                const float dhw = w * dh;
                float h;
                if (C::kPairB) {
                  const float uu = __uint_as_float(u[2 * j + b]);
                  const float sg = sigmoid_fast(zz);
                  h = zz * sg * uu;
                  vz[b] = dhw * uu * sg * (1.0f + zz * (1.0f - sg));
                  vu[b] = dhw * zz * sg;
                } else {
                  const float sg = gelu_gate(zz);
                  h = zz * sg;
                  vz[b] = dhw * (sg + zz * sg * (1.0f - sg) * 2.0f * kGeluC * (1.0f + 3.0f * 0.044715f * zz * zz));
                  vu[b] = 0.0f;
                }
                vh[b] = w * h;
                dot += dh * h;  // columns behind N1 hold zeros
                if (!live) vz[b] = vu[b] = vh[b] = 0.0f;
              }
              pz[i0 / 2 + j] = pack2(vz[0], vz[1]);
              pu[i0 / 2 + j] = pack2(vu[0], vu[1]);
              ph[i0 / 2 + j] = pack2(vh[0], vh[1]);
            }
          }
          // all 128 rows of the CTA's tile: the weight gradients read zeros behind the last one
          const int all = q.rows > 128 * rank ? 32 : 0;
          uint8_t* dz = reinterpret_cast<uint8_t*>(a.out) + slot0 * pitch + (int64_t)n * 2;
          store_rows<4>(stage, pz, dz, pitch, all, (a.N - n) / 8, lane);
          if (C::kPairB) store_rows<4>(stage, pu, dz + (int64_t)a.N * 2, pitch, all, (a.N - n) / 8, lane);
          store_rows<4>(stage, ph, reinterpret_cast<uint8_t*>(a.out2) + (slot0 * a.N + n) * 2, (int64_t)a.N * 2, all,
                        (a.N - n) / 8, lane);
        }
        if (live) a.part[slot * (2 * a.col_tiles) + 2 * (q.n0 / C::kOutCols) + half] = dot;
      } else {
        const int64_t m = (int64_t)q.m0 + r0;
        uint8_t* base = reinterpret_cast<uint8_t*>(a.out) + (((int64_t)q.e * a.M + m) * a.N + q.n0) * 2;
#pragma unroll 1
        for (int c = half * 32; c < BN; c += 64) {
          uint32_t z[32], p[16];
          if (empty_tile) {
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] = 0;
          } else {
            ptx::tmem_ld_32x32b_x32(d + c, z);
            ptx::tmem_ld_wait();
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) p[i] = pack2(__uint_as_float(z[2 * i]), __uint_as_float(z[2 * i + 1]));
          store_rows<4>(stage, p, base + c * 2, (int64_t)a.N * 2, (int)(a.M - m), (a.N - q.n0 - c) / 8, lane);
        }
      }
      if (!empty_tile) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) ptx::mbar_arrive(&tempty[buf]);
          else ptx::mbar_arrive_cluster(ptx::mapa(&tempty[buf], 0));
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (PAIR == 2) ptx::cluster_sync();  // both CTAs are done with the pair's TMEM and barriers
  if (warp == 1) {
    ptx::tc_fence_after();
    if (PAIR == 2) ptx::tmem_dealloc_pair(tmem, C::kTmemCols);
    else ptx::tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace moe
}  // namespace cusync
