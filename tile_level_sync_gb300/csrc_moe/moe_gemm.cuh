// The products of an expert layer: one persistent tcgen05 kernel per product.
//
// Products over slots (tokens in dispatch order) are computed transposed: the MMA's 128
// rows (256 across a pair of CTAs, cta_group::2) are columns of the expert's weights, its
// columns are the tile's tokens.  The width then follows the expert's rows in steps of 16 (32),
// where tiles of 128 or 256 token rows would be filled up with rows that count for nothing
// (4096 tokens x 8 of 64 experts: a quarter of the work), and a lane of the accumulator is
// an output column, so that a warp stores 32 neighbours of a token's row at once.
//
//   mode   A (M)                      B (N)                  epilogue
//   FWD1   W1t[e] rows (G * N1)       X by slot              h = act(z), bf16
//   FWD1G  the same                   X (gather)
//   FWD2   W2t[e] rows (D)            H                      O, fp16 scaled by slot and 32 columns
//   BWD1   W1t[e] gate, up;           X; dY by slot          dZ and w h, bf16; sums of dH h
//          W2t[e] along N1
//   DX     W1t[e] along D             dZ                     dX per slot, as O
//   DW     dZ along G * N1            X along D              dW1t[e], bf16   (K = slots), then
//          dY along D                 w h along N1           dW2t[e], bf16
//
// "along": the operand is stored with its M (or N) index contiguous rather than K, and the
// MMA reads it that way, so nothing is ever transposed in memory.  FWD1's SwiGLU tile
// takes gate and up rows of W1t eight by eight (one 5-D box): a gate lane and the lane
// eight further hold the two factors of one h.  BWD1 has them in accumulators of their own.
//
// One CTA (or pair) per SM.  Tiles differ in length, so they are claimed one by one from a
// counter that the plan cleared; the claim of a tile is made when the one before it starts, or
// the one before that where tiles are short and a claim (2 us) would be waited for:
//   last warp  (of a pair's first CTA) claims tiles, reads their plan entries and hands them
//              to the other warps of both CTAs through a ring in shared memory.
//   warp 0     copies of A, the last warp but one copies of B (TMA boxes; FWD1G: tile::gather4, four
//              rows a copy, through the plan's row indices).  A copy has a fixed cost
//              besides its bytes, so a stage holds two blocks of 64 k where three such
//              stages fit, and where widths allow one box brings all of an operand.
//   warp 1     TMEM owner; lane 0 (of a pair's first CTA) issues tcgen05.mma.  In a pair's second CTA
//              it hands the accumulators that the epilogue there has read back to the first, and
//              the last warp the ring's slots: arrivals across the pair need a release, which waits for
//              the thread's own stores, and these two warps have none (the weight gradients'
//              epilogue took 5200 cycles a tile in the second CTA, 3000 in the first, when it
//              made them itself).
//   warps 2 .. epilogue: two (BWD1: four) warps per TMEM lane quarter, 32 (16) columns each in
//              turn.
// Accumulators are double-buffered where two fit in TMEM's 512 columns.
//
// X by slot is a copy in dispatch order (dispatch_kernel).  The gather needs none, but
// brings 128 rows x 64 columns in 1.25 us, more than twice what their MMAs take: it is for
// tiles of few rows.
//
// O and dX per slot are sums over a token's experts in fp32 still to be made: their 16 bits
// are fp16 with a power of two for every slot and 32 columns, at half the bytes of fp32: at most
// 2^-11 of a value off, where it is above 2^-29 of the slot's largest of the 32, beside the 2^-8 of
// the bf16 result.  One power for 32 slots together saves 2 us of 379 (4096 tokens), but takes the
// bits of a token that stands beside one 2^30 times as large.
//
// Token rows behind an expert's last one are columns of their own and are not stored.  In
// the weight gradients K runs over slots in steps of 16: dispatch_kernel and BWD1 store
// zeros up to the step's end.
//
// Both weights' gradients are one launch, whose second half fills the first's tail: 12 us less
// of 378 for 4096 tokens, 8 of 84 in the gradient of 333 tokens.
//
// Every wait is bounded; an expired one raises the error word and ends the CTA's roles.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "moe_plan.cuh"
#include "moe_ptx.cuh"

namespace cusync {
namespace moe {

enum : int { FWD1 = 0, FWD2 = 1, BWD1 = 2, DX = 3, DW = 4, FWD1G = 5 };

constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kTileSlots = 4;
constexpr int kRowStep = 16;                 // slots up to a multiple of which a row's zeros are stored
constexpr uint32_t kErrWait = 3u << 24;      // the pipeline-wait class of the chain kernel's error words

struct GemmArgs {
  CUtensorMap mA;      // weights; DW: dZ
  CUtensorMap mA2;     // BWD1: W2t; DW: dY
  CUtensorMap mB[4];   // tokens, boxes of 16, 32, 64 and 128 (BWD1 on pairs: 80) rows (gather: [0],
                       // one row); DW: [0], X
  CUtensorMap mB2[4];  // BWD1: dY; DW: [0], w H
  CUtensorMap mO;      // the output, boxes of 32 rows x a warp's columns; BWD1: dZ, 16 x 32;
                       // DW: dW1t
  CUtensorMap mO2;     // BWD1: w H; DW: dW2t
  int32_t* plan;
  const float* weights;
  void* out;           // H, O or dX per slot
  uint8_t* scale;      // FWD2, DX: exponents of the slots' blocks of 32 columns (scale_at)
  float* part;         // BWD1: sums of dH h over 32 columns of N1, [slot][parts]
  int64_t counts, offsets, tiles, row_of;  // plan words; tiles: of the launch's 128, 160 or 256 rows
  int32_t T, k, E;
  int32_t M;           // output columns (DW: rows of an expert's matrix)
  int32_t N;           // DW: output columns
  int32_t K;           // reduction length (not DW)
  int32_t m_tiles, n_tiles, parts, slots;
  int32_t M2, N2, m_tiles2, n_tiles2;  // DW: of dW2t
  int32_t counter;     // plan word that counts this launch's claimed tiles
  // Every width is a multiple of 64: the maps see rows as [width / 64][rows][64], and one
  // copy brings an operand's two blocks of 64 k, or its two chunks of 64 columns, at once.
  int32_t wide;
};

template <int MODE, int ACT, int PAIR>
struct GemmCfg {
  static constexpr bool kDw = MODE == DW;
  static constexpr bool kBwd1 = MODE == BWD1;
  static constexpr bool kFwd1 = MODE == FWD1 || MODE == FWD1G;
  static constexpr bool kGather = MODE == FWD1G;
  static constexpr bool kGated = ACT == 1 && kFwd1;        // gate and up rows eight by eight
  static constexpr bool kMnA = kDw || MODE == DX;
  static constexpr int kG = ACT == 1 ? 2 : 1;
  static constexpr int kAParts = kBwd1 ? kG + 1 : 1;       // 128 x 64 blocks of A in a stage
  static constexpr int kBParts = kBwd1 ? 2 : 1;
  // widest tile: BWD1's three accumulators leave room for 160 columns
  static constexpr int kCols = kDw ? 256 : PAIR == 1 ? 128 : kBwd1 ? 160 : 256;
  static constexpr int kTileCount = kCols == 256 ? PLAN_PAIRS : kCols == 160 ? PLAN_MIDS : PLAN_TILES;
  static constexpr int kLastBox = kCols / PAIR;            // rows of the highest token box
  static constexpr int kColStep = 16 * PAIR;               // of the MMA's width
  static constexpr int kBBytes = kCols / PAIR * 128;       // a CTA's share of B
  static constexpr int kABytes = 128 * 128;
  static constexpr int kBlockBytes = kAParts * kABytes + kBParts * kBBytes;  // 64 k
  static constexpr int kKps = kBlockBytes <= 32 * 1024 ? 2 : 1;              // blocks of 64 k in a stage
  static constexpr int kStageBytes = kKps * kBlockBytes;
  // Epilogue warps, a multiple of four.  BWD1 has no second set of accumulators to hide its
  // epilogue behind: twice the warps.
  static constexpr int kEpi = kBwd1 ? 16 : 8;
  static constexpr int kThreads = (kEpi + 4) * 32;
  // Outputs by slot: on pairs (BWD1: always) staged in shared memory and stored by TMA, 32 (16) rows at a time; on
  // single CTAs, whose tiles often have few rows, stored from registers, real rows only.
  static constexpr bool kStaged = PAIR == 2 && (kFwd1 || MODE == FWD2 || MODE == DX);
  static constexpr int kRing = (kDw || kStaged ? 192 : 224) * 1024;
  static constexpr int kStages = kRing / kStageBytes < 8 ? kRing / kStageBytes : 8;
  // epilogue: two blocks of 2 KB a warp; BWD1 one of 1 KB
  static constexpr int kWarpOut = kBwd1 ? 1024 : kDw || kStaged ? 4096 : 0;
  static constexpr int kStageOut = kEpi * kWarpOut;
  static constexpr int kAccCols = kAParts * kCols;
  static constexpr int kAccs = 2 * kAccCols <= 512 ? 2 : 1;
  static constexpr int kTmemCols = kAccs * kAccCols <= 256 ? 256 : 512;
  static_assert(kAccs * kAccCols <= 512, "TMEM columns");
  static constexpr int kFeatures = (kGated ? 64 : 128) * PAIR;  // output columns of a tile (DW: rows)
  static constexpr int kSmemBytes = kStages * kStageBytes + kStageOut + 1024;
};

// Where the exponent of a slot's block of 32 columns is: those of 256 columns beside each other,
// as a warp of combine_kernel reads them.
__host__ __device__ __forceinline__ int64_t scale_at(int64_t slots, int64_t slot, int block) {
  return ((block / 8) * slots + slot) * 8 + block % 8;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store_bf16(uint16_t* p, float v) {
  *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
// 1 / (1 + e^-x); the fast exponential and division are within a few 1e-7 of it
__device__ __forceinline__ float sigmoid_fast(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// The same to some ulp, where 32 bits of the result count (dweights): expf within 2, the division
// within 2
__device__ __forceinline__ float sigmoid_full(float x) { return __fdividef(1.0f, 1.0f + expf(-x)); }

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
// The argument of the sigmoid in GeLU_tanh(z) = z sigmoid(2 c (z + 0.044715 z^3)), and that sigmoid
__device__ __forceinline__ float gelu_arg(float z) { return 2.0f * kGeluC * (z + 0.044715f * z * z * z); }
__device__ __forceinline__ float gelu_gate(float z) { return sigmoid_fast(gelu_arg(z)); }

// One tile of a launch: `rows` tokens of expert e from slot0 on (DW: all of the expert's),
// output columns (DW: matrix rows) from m0 on, DW: columns from n0 on; nkb blocks of 64 k.  DW
// computes both weights' gradients: from e = E on dW2t of expert e - E.
struct Tile {
  int32_t e, slot0, rows, m0, n0, nkb;
};

template <int MODE, int ACT, int PAIR>
__device__ __forceinline__ int32_t tile_total(const GemmArgs& a) {
  if (GemmCfg<MODE, ACT, PAIR>::kDw) return a.E * (a.m_tiles * a.n_tiles + a.m_tiles2 * a.n_tiles2);
  return a.plan[GemmCfg<MODE, ACT, PAIR>::kTileCount] * a.m_tiles;
}

template <int MODE, int ACT, int PAIR>
__device__ __forceinline__ Tile tile_at(const GemmArgs& a, int32_t t) {
  using C = GemmCfg<MODE, ACT, PAIR>;
  Tile r;
  if (C::kDw) {
    const int32_t first = a.E * a.m_tiles * a.n_tiles;  // tiles of dW1t
    const bool second = t >= first;
    if (second) t -= first;
    const int32_t m_tiles = second ? a.m_tiles2 : a.m_tiles, per = m_tiles * (second ? a.n_tiles2 : a.n_tiles);
    const int32_t e = t / per, q = t - e * per;
    r.e = second ? a.E + e : e;
    r.m0 = (q % m_tiles) * C::kFeatures;
    r.n0 = (q / m_tiles) * C::kCols;
    r.slot0 = a.plan[a.offsets + e];
    r.rows = a.plan[a.counts + e];
    r.nkb = (r.rows + 63) / 64;
  } else {
    const int32_t rt = t / a.m_tiles;
    const int4 er = *reinterpret_cast<const int4*>(a.plan + a.tiles + 4 * rt);
    r.e = er.x;
    r.slot0 = er.y;
    r.rows = er.z;
    r.m0 = (t - rt * a.m_tiles) * C::kFeatures;
    r.n0 = 0;
    r.nkb = (a.K + 63) / 64;
  }
  return r;
}

// The ring of claimed tiles.  full: one arrival by the claiming warp; empty: arrivals by every
// warp of the CTA that read the slot, and in a pair's first CTA one for all of the second's; each
// CTA has its own.  taken (the first CTA's): an arrival by the first copying warp alone.
struct TileRing {
  int32_t slot[kTileSlots][8];  // a Tile; rows < 0: no more
  uint64_t full[kTileSlots], empty[kTileSlots], taken[kTileSlots];
};

// One warp's way through the ring.
template <int PAIR>
struct Walk {
  TileRing& ring;
  uint32_t n;
  __device__ __forceinline__ explicit Walk(TileRing& r) : ring(r), n(0) {}
  // The next tile, in every lane.  False at the end, and (with *ok cleared) if a wait expired.
  __device__ __forceinline__ bool take(Tile& q, bool* ok, bool first_copier = false) {
    const uint32_t s = n % kTileSlots, par = (n / kTileSlots) & 1;
    const bool got = PAIR == 2 ? ptx::mbar_wait_bounded_cluster(&ring.full[s], par, kWaitNs)
                               : ptx::mbar_wait_bounded(&ring.full[s], par, kWaitNs);
    if (!__all_sync(0xffffffffu, got)) {
      *ok = false;
      return false;
    }
    const volatile int32_t* v = ring.slot[s];
    const int lane = threadIdx.x & 31;
    const int32_t mine = v[lane & 7];
    // broadcast, so that what is computed from the tile is known to be uniform
    q.e = __shfl_sync(0xffffffffu, mine, 0);
    q.slot0 = __shfl_sync(0xffffffffu, mine, 1);
    q.rows = __shfl_sync(0xffffffffu, mine, 2);
    q.m0 = __shfl_sync(0xffffffffu, mine, 3);
    q.n0 = __shfl_sync(0xffffffffu, mine, 4);
    q.nkb = __shfl_sync(0xffffffffu, mine, 5);
    if (lane == 0) {
      ptx::mbar_arrive(&ring.empty[s]);
      if (first_copier) ptx::mbar_arrive(&ring.taken[s]);
    }
    __syncwarp();
    ++n;
    return q.rows >= 0;
  }
};

// A warp's two blocks of 2 KB in turn for TMA stores: the block to fill, once the store before
// the last has read it ...
__device__ __forceinline__ uint16_t* stage_block(uint8_t* stage, uint32_t blocks) {
  if ((threadIdx.x & 31) == 0) ptx::bulk_wait_group_read<1>();
  __syncwarp();
  return reinterpret_cast<uint16_t*>(stage + (blocks % 2) * 2048);
}
// ... and its store: to columns from c0, rows from r0 of matrix e on; or, without e, to columns
// from c0, slots from r0 on.  Slots behind an expert's last row are written too: up to its next
// multiple of 32 they are no one else's, and no one's input but to columns of their own.
__device__ __forceinline__ void store_block(const CUtensorMap* m, uint8_t* stage, uint32_t& blocks, int32_t c0,
                                            int32_t r0, int32_t e = -1) {
  ptx::fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    if (e < 0) ptx::tma_store_2d(m, stage + (blocks % 2) * 2048, c0, r0);
    else ptx::tma_store_3d(m, stage + (blocks % 2) * 2048, c0, r0, e);
    ptx::bulk_commit_group();
  }
  ++blocks;
}

// Sums over the warp's lanes of 16 values: lanes i and i + 16 end with the sum of v[i].
__device__ __forceinline__ float transpose_sum(float (&v)[16], int lane) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
#pragma unroll
  for (int o = 8; o; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = up ? v[i + o] : v[i], send = up ? v[i] : v[i + o];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return v[0];
}

template <int MODE, int ACT, int PAIR>
__global__ void __launch_bounds__(GemmCfg<MODE, ACT, PAIR>::kThreads, 1) moe_gemm_kernel(const __grid_constant__ GemmArgs a) {
  using C = GemmCfg<MODE, ACT, PAIR>;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t full[C::kStages], empty[C::kStages], tfull[2], tempty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int32_t abort_flag;
  __shared__ TileRing tiles;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = PAIR == 2 ? (int)ptx::cluster_ctarank() : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&tfull[i], 1);
      ptx::mbar_init(&tempty[i], C::kEpi + (PAIR == 2 && rank == 0));  // and the other CTA's warp 1
    }
    ptx::mbar_init(&drain, 1);
    for (int i = 0; i < kTileSlots; ++i) {
      ptx::mbar_init(&tiles.full[i], 1);
      // copies, warp 1, epilogue, and the last warp: the second CTA's own, the first CTA's for those
      ptx::mbar_init(&tiles.empty[i], C::kEpi + (PAIR == 2 ? 4 : 3));
      ptx::mbar_init(&tiles.taken[i], 1);
    }
    ptx::mbar_init_fence();
    abort_flag = 0;
    ptx::prefetch_tmap(&a.mA);
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
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  Walk<PAIR> walk(tiles);
  Tile q;

  if (warp == 0 || warp == C::kEpi + 2) {
    // ------------------------------------------------------------ copies
    const bool copies_a = warp == 0;
    const uint64_t pol = ptx::l2_policy_evict_normal();
    const bool one = ptx::elect_one();
    uint32_t it = 0, st = 0, par = 1;
    const uint32_t full0 = PAIR == 2 ? ptx::mapa(&full[0], 0) : 0;
    bool ok = true;
    while (!abort_flag && walk.take(q, &ok, copies_a && rank == 0)) {
      // this CTA's share of the tile's tokens, and the box that covers it
      const int cols = C::kDw ? C::kCols : (q.rows + C::kColStep - 1) / C::kColStep * C::kColStep;
      const int share = cols / PAIR;
      const int pick = share <= 16 ? 0 : share <= 32 ? 1 : share <= 64 ? 2 : 3;
      const bool second = C::kDw && q.e >= a.E;
      const CUtensorMap* ma = second ? &a.mA2 : &a.mA;
      const CUtensorMap *mb = C::kDw ? (second ? &a.mB2[0] : &a.mB[0]) : &a.mB[pick], *mb2 = &a.mB2[pick];
      const int32_t slot = q.slot0 + rank * share;
      const int32_t m0 = q.m0 + rank * (C::kFeatures / PAIR), n0 = q.n0 + rank * (C::kCols / PAIR);
      // a lane's four gathered rows, as token indices; -1 (a slot behind the last row)
      // becomes T, outside the tensor, read as zero
      const int live = C::kGather ? (q.rows + 3) / 4 : 0;
      int4 tok = make_int4(a.T, a.T, a.T, a.T);
      if (C::kGather && !copies_a && lane < live) {
        const int4 r = *reinterpret_cast<const int4*>(a.plan + a.row_of + q.slot0 + 4 * lane);
        auto token = [&](int32_t x) { return x < 0 ? a.T : x / a.k; };
        tok = make_int4(token(r.x), token(r.y), token(r.z), token(r.w));
      }
      const uint32_t b_bytes = C::kGather ? live * 512 : C::kDw ? C::kBBytes : (pick == 3 ? C::kLastBox : 16 << pick) * 128;
      const uint32_t block_bytes = PAIR * (C::kAParts * C::kABytes + C::kBParts * b_bytes);
      // Nothing orders the two warps' copies: the barrier's phase cannot end before warp 0's
      // arrival.
      for (int kb0 = 0; kb0 < q.nkb; kb0 += C::kKps, ++it) {
        ok = ptx::mbar_wait_bounded(&empty[st], par, kWaitNs);
        if (!ok) break;
        uint8_t* sA = ring + st * C::kStageBytes;
        uint8_t* sB = sA + C::kKps * C::kAParts * C::kABytes;
        uint64_t* bar = &full[st];
        // in a pair both CTAs' copies complete on the first one's barrier
        const uint32_t bar0 = full0 + 8 * st;
        auto load2 = [&](void* dst, const CUtensorMap* m, int32_t c0, int32_t c1) {
          if (PAIR == 2) ptx::tma_load_2d_to_leader(dst, m, bar0, c0, c1, pol);
          else ptx::tma_load_2d(dst, m, bar, c0, c1, pol);
        };
        auto load3 = [&](void* dst, const CUtensorMap* m, int32_t c0, int32_t c1, int32_t c2) {
          if (PAIR == 2) ptx::tma_load_3d_to_leader(dst, m, bar0, c0, c1, c2, pol);
          else ptx::tma_load_3d(dst, m, bar, c0, c1, c2, pol);
        };
        auto load5 = [&](void* dst, const CUtensorMap* m, int32_t c0, int32_t c3, int32_t c4) {
          if (PAIR == 2) ptx::tma_load_5d_to_leader(dst, m, bar0, c0, 0, 0, c3, c4, pol);
          else ptx::tma_load_5d(dst, m, bar, c0, 0, 0, c3, c4, pol);
        };
        if (++st == C::kStages) {
          st = 0;
          par ^= 1;
        }
        const bool wide = a.wide;
        const int blocks = min(C::kKps, q.nkb - kb0);
        if (copies_a && rank == 0 && one) {
          // a box of two blocks counts whole where the second lies outside
          const int counted = wide && !C::kGather ? C::kKps : blocks;
          ptx::mbar_arrive_expect_tx(bar, C::kGather && wide ? C::kKps * C::kABytes + blocks * b_bytes
                                                             : counted * block_bytes);
        }
        if (wide && copies_a) {
          const int32_t kc = kb0 * 64;
          if (one) {
            if (C::kDw) {
              load3(sA, ma, 0, q.slot0 + kc, m0 / 64);
            } else if (C::kGated) {
              load5(sA, &a.mA, 0, q.e * (2 * a.M / 8) + m0 / 8, kb0);
            } else if (C::kBwd1) {
              load3(sA, &a.mA, kc, q.e * C::kG * a.M + m0, 0);
              load3(sA + C::kG * C::kABytes, &a.mA2, 0, q.e * a.K + kc, m0 / 64);
            } else if (MODE == DX) {
              load3(sA, &a.mA, 0, q.e * a.K + kc, m0 / 64);
            } else {
              load3(sA, &a.mA, 0, q.e * a.M + m0, kb0);
            }
          }
        } else if (wide && !C::kGather) {
          const int32_t kc = kb0 * 64;
          if (one) {
            if (C::kDw) {
              load3(sB, mb, 0, q.slot0 + kc, n0 / 64);
              if (PAIR == 1) load3(sB + 2 * C::kKps * 8192, mb, 0, q.slot0 + kc, n0 / 64 + 2);
            } else {
              load3(sB, mb, 0, slot, kb0);
              if (C::kBwd1) load3(sB + C::kBBytes, mb2, 0, slot, kb0);
            }
          }
        } else {
#pragma unroll
          for (int b = 0; b < C::kKps; ++b) {
            if (b >= blocks) break;
            uint8_t* pA = sA + b * C::kABytes;
            uint8_t* pB = sB + b * C::kBBytes;
            const int32_t kc = (kb0 + b) * 64;
            if (copies_a) {
              if (one) {
                if (C::kDw) {
                  load2(pA, ma, m0, q.slot0 + kc);
                  load2(pA + 8192, ma, m0 + 64, q.slot0 + kc);
                } else if (C::kGated) {
                  load5(pA, &a.mA, kc, m0 / 8, q.e);
                } else if (C::kBwd1) {
                  load3(pA, &a.mA, kc, m0, C::kG * q.e);
                  if (C::kG == 2) load3(pA + C::kABytes, &a.mA, kc, m0, 2 * q.e + 1);
                  load3(pA + C::kG * C::kABytes, &a.mA2, m0, kc, q.e);
                  load3(pA + C::kG * C::kABytes + 8192, &a.mA2, m0 + 64, kc, q.e);
                } else if (MODE == DX) {
                  load3(pA, &a.mA, m0, kc, q.e);
                  load3(pA + 8192, &a.mA, m0 + 64, kc, q.e);
                } else {
                  load3(pA, &a.mA, kc, m0, q.e);
                }
              }
            } else if (C::kGather) {
              if (lane < live) ptx::tma_gather4(pB + lane * 512, mb, bar, kc, tok, pol);
            } else if (one) {
              if (C::kDw) {
#pragma unroll
                for (int c = 0; c < C::kCols / PAIR / 64; ++c) load2(pB + c * 8192, mb, n0 + 64 * c, q.slot0 + kc);
              } else {
                load2(pB, mb, kc, slot);
                if (C::kBwd1) load2(pB + C::kBBytes, mb2, kc, slot);
              }
            }
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
    }
    if (!ok && lane == 0) {
      abort_flag = 1;
      a.plan[PLAN_ERR] = (int32_t)kErrWait;
    }
    __syncwarp();
    // after an abort: wait, bounded, for the copies still in flight (both warps' complete on `full`)
    if (abort_flag && copies_a && lane == 0 && rank == 0)
      for (uint32_t i = it > (uint32_t)C::kStages ? it - C::kStages : 0; i < it; ++i)
        ptx::mbar_wait_bounded(&full[i % C::kStages], (i / C::kStages) & 1, kWaitNs);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (rank == 0) {
      auto mma = [&](uint32_t d, uint64_t da, uint64_t db, uint32_t id, uint32_t more) {
        if (PAIR == 2) ptx::umma_bf16_pair(d, da, db, id, more);
        else ptx::umma_bf16(d, da, db, id, more);
      };
      auto commit = [&](uint64_t* bar) {
        if (PAIR == 2) ptx::umma_commit_pair_multicast(bar, 0x3);
        else ptx::umma_commit(bar);
      };
      const uint32_t ring0 = __shfl_sync(0xffffffffu, ptx::smem_u32(ring), 0);
      const bool one = ptx::elect_one();  // the lane whose MMAs its commits cover
      const bool wide = a.wide;
      const uint32_t chunk = wide ? C::kKps * 8192 : 8192;  // 64 columns of an operand that lies along M or N
      uint32_t st = 0, par = 0, acc = 0;
      bool ok = true;
      while (ok && !abort_flag && walk.take(q, &ok)) {
        if (q.nkb == 0) continue;  // an expert without rows: the epilogue writes zeros
        const uint32_t cols = C::kDw ? C::kCols : (q.rows + C::kColStep - 1) / C::kColStep * C::kColStep;
        const uint32_t share = cols / PAIR;
        const uint32_t box_bytes = (share <= 16 ? 16 : share <= 32 ? 32 : share <= 64 ? 64 : C::kLastBox) * 128;
        const uint32_t idesc = ptx::idesc_bf16_f32(128 * PAIR, cols) | (C::kMnA ? ptx::kIdescAMn : 0) |
                               (C::kDw ? ptx::kIdescBMn : 0);
        const uint32_t buf = acc % C::kAccs, use = acc / C::kAccs;
        ++acc;
        ok = (PAIR == 2 ? ptx::mbar_wait_bounded_cluster(&tempty[buf], (use & 1) ^ 1, kWaitNs)
                        : ptx::mbar_wait_bounded(&tempty[buf], (use & 1) ^ 1, kWaitNs)) &&
             !abort_flag;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem + buf * C::kAccCols;
        for (int kb0 = 0; kb0 < q.nkb; kb0 += C::kKps) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(&full[st], par, kWaitNs));
          if (!ok) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int b = 0; b < C::kKps; ++b) {
            const int kb = kb0 + b;
            // block b of the stage: wide boxes put a chunk's blocks, and a token box's, back to back
            const uint32_t st0 = ring0 + st * C::kStageBytes;
            const uint32_t sA = st0 + b * (C::kMnA && wide ? 8192 : C::kABytes);
            const uint32_t sB = st0 + C::kKps * C::kAParts * C::kABytes +
                                b * (C::kDw && wide ? 8192 : wide && !C::kGather ? box_bytes : C::kBBytes);
            // 16 k: 32 bytes of a K-contiguous row, or 16 rows of 128 bytes
            constexpr uint64_t mn = 2048 >> 4, kk = 32 >> 4;
            const uint64_t dA = C::kMnA ? ptx::smem_desc_mn128(sA, chunk) : ptx::smem_desc_k128(sA);
            const uint64_t dB = C::kDw ? ptx::smem_desc_mn128(sB, chunk) : ptx::smem_desc_k128(sB);
            const uint64_t dA2 = ptx::smem_desc_mn128(sA + C::kG * C::kABytes, 8192);
            const uint64_t dB2 = ptx::smem_desc_k128(sB + C::kBBytes);
            // the last block's steps of 16: only those that hold k (DW: rows; elsewhere columns)
            const int left = (C::kDw ? q.rows : a.K) - kb * 64;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              if (16 * s >= left) break;
              if (!one) continue;
              if (C::kBwd1) {
#pragma unroll
                for (int p = 0; p < C::kG; ++p)
                  mma(d + p * C::kCols, dA + p * (C::kABytes >> 4) + s * kk, dB + s * kk, idesc, kb || s);
                mma(d + C::kG * C::kCols, dA2 + s * mn, dB2 + s * kk, idesc | ptx::kIdescAMn, kb || s);
              } else {
                mma(d, dA + s * (C::kMnA ? mn : kk), dB + s * (C::kDw ? mn : kk), idesc, kb || s);
              }
            }
          }
          if (one) commit(&empty[st]);
          __syncwarp();
          if (++st == C::kStages) {
            st = 0;
            par ^= 1;
          }
        }
        if (!ok) break;
        if (one) commit(&tfull[buf]);
        __syncwarp();
      }
      if (!ok || abort_flag) {
        abort_flag = 1;
        a.plan[PLAN_ERR] = (int32_t)kErrWait;
        if (one) commit(&drain);  // MMAs still in flight
        ptx::mbar_wait_bounded(&drain, 0, kWaitNs);
      }
    } else {
      // a pair's second CTA: accumulators back to the first as the epilogue here is done with them
      uint32_t acc = 0;
      bool ok = true;
      while (!abort_flag && walk.take(q, &ok)) {
        if (q.nkb == 0) continue;
        const uint32_t buf = acc % C::kAccs, use = acc / C::kAccs;
        ++acc;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(&tempty[buf], use & 1, kWaitNs));
        if (!ok) break;
        if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa(&tempty[buf], 0));
        __syncwarp();
      }
      if (!ok) {
        abort_flag = 1;
        a.plan[PLAN_ERR] = (int32_t)kErrWait;
      }
    }
    __syncwarp();
  } else if (warp == C::kEpi + 3) {
    // ------------------------------------------------------------ claims
    if (rank == 0 && lane == 0) {
      const int32_t total = tile_total<MODE, ACT, PAIR>(a);
      const uint32_t ahead = C::kDw ? 3 : a.K < 24 * 64 ? 2 : 1;
      bool ok = true;
      for (uint32_t n = 0; !abort_flag; ++n) {
        const uint32_t s = n % kTileSlots;
        if (n >= kTileSlots)
          ok = PAIR == 2 ? ptx::mbar_wait_bounded_cluster(&tiles.empty[s], ((n / kTileSlots) & 1) ^ 1, kWaitNs)
                         : ptx::mbar_wait_sleepy(&tiles.empty[s], ((n / kTileSlots) & 1) ^ 1, kWaitNs);
        if (ok && n >= ahead) {
          const uint32_t before = n - ahead;
          ok = ptx::mbar_wait_bounded(&tiles.taken[before % kTileSlots], (before / kTileSlots) & 1, kWaitNs);
        }
        if (!ok) break;
        int32_t t = blockIdx.x / PAIR;  // the first tile needs no claim
        if (n) t = gridDim.x / PAIR + atomicAdd(a.plan + a.counter, 1);
        Tile q = {0, 0, -1, 0, 0, 0};
        if (t < total) q = tile_at<MODE, ACT, PAIR>(a, t);
        const int32_t v[6] = {q.e, q.slot0, q.rows, q.m0, q.n0, q.nkb};
#pragma unroll
        for (int i = 0; i < 6; ++i) {
          *const_cast<volatile int32_t*>(&tiles.slot[s][i]) = v[i];
          if (PAIR == 2) ptx::st_cluster_u32(ptx::mapa(&tiles.slot[s][i], 1), (uint32_t)v[i]);
        }
        ptx::mbar_arrive(&tiles.full[s]);
        if (PAIR == 2) ptx::mbar_arrive_cluster(ptx::mapa(&tiles.full[s], 1));
        if (t >= total) break;
      }
      if (!ok) {
        abort_flag = 1;
        a.plan[PLAN_ERR] = (int32_t)kErrWait;
      }
    } else if (rank == 1) {
      // the ring's slots back to the claiming warp as all of this CTA's warps have read them
      bool ok = true;
      for (uint32_t n = 0; !abort_flag && walk.take(q, &ok); ++n) {
        const uint32_t s = n % kTileSlots;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(&tiles.empty[s], (n / kTileSlots) & 1, kWaitNs));
        if (!ok) break;
        if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa(&tiles.empty[s], 0));
        __syncwarp();
      }
      if (!ok) {
        abort_flag = 1;
        a.plan[PLAN_ERR] = (int32_t)kErrWait;
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;               // TMEM lane quarter
    constexpr int cols = C::kBwd1 ? 16 : 32;    // columns at a time
    const int first = ((warp - 2) >> 2) * cols;  // this warp's first, and from there to its next
    constexpr int step = C::kEpi / 4 * cols;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    uint8_t* stage = ring + C::kStages * C::kStageBytes + (warp - 2) * C::kWarpOut;
    uint32_t acc = 0, blocks = 0;
    bool ok = true;
    while (walk.take(q, &ok)) {
      const bool empty_tile = q.nkb == 0;
      const uint32_t buf = acc % C::kAccs, use = acc / C::kAccs;
      // BWD1: the weights of this warp's tokens, while the product runs: of its first 16 in lanes
      // 0 to 15, of the next in the others, of the third in w_held[1]
      float w_held[2] = {0.0f, 0.0f};
      if (C::kBwd1) {
        static_assert(!C::kBwd1 || C::kCols <= 4 * step, "a warp's tokens fit w_held");
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = first + (2 * h + lane / 16) * step + lane % 16;
          const int r = c < q.rows ? a.plan[a.row_of + q.slot0 + c] : -1;
          if (r >= 0) w_held[h] = a.weights[r];
        }
      }
      if (!empty_tile) {
        ++acc;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_sleepy(&tfull[buf], use & 1, kWaitNs) && !abort_flag);
        if (!ok) break;
        ptx::tc_fence_after();
      }
      const uint32_t d = tmem + buf * C::kAccCols + lanes;
      const int lane0 = 128 * rank + quarter * 32;  // this warp's first accumulator lane in the tile
      if (C::kGated) {
        // lanes 0-7 and 16-23 hold gate values, the lanes eight further the up values of the
        // same column of H; of two tokens each of the two lanes computes one
        const int up = (lane >> 3) & 1, own = (lane >> 4) * 8 + (lane & 7);
#pragma unroll 1
        for (int c = first; c < q.rows; c += step) {
          uint32_t z[32];
          ptx::tmem_ld_32x32b_x32(d + c, z);
          ptx::tmem_ld_wait();
          const int f = q.m0 + lane0 / 2 + own, left = f < a.M ? q.rows - c - up : 0;
          uint16_t* out = C::kStaged ? stage_block(stage, blocks) + up * 16 + own
                                     : reinterpret_cast<uint16_t*>(a.out) + (int64_t)(q.slot0 + c + up) * a.M + f;
          const int64_t pitch = C::kStaged ? 16 : a.M;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float z0 = __uint_as_float(z[2 * i]), z1 = __uint_as_float(z[2 * i + 1]);
            const float other = __shfl_xor_sync(0xffffffffu, up ? z0 : z1, 8);
            const float g = up ? other : z0, u = up ? z1 : other;
            if (C::kStaged || 2 * i < left) store_bf16(out + 2 * i * pitch, g * sigmoid_fast(g) * u);
          }
          if (C::kStaged) store_block(&a.mO, stage, blocks, q.m0 + lane0 / 2, q.slot0 + c);
        }
      } else if (C::kFwd1) {
#pragma unroll 1
        for (int c = first; c < q.rows; c += step) {
          uint32_t z[32];
          ptx::tmem_ld_32x32b_x32(d + c, z);
          ptx::tmem_ld_wait();
          const int f = q.m0 + lane0 + lane, left = f < a.M ? q.rows - c : 0;
          uint16_t* out = C::kStaged ? stage_block(stage, blocks) + lane
                                     : reinterpret_cast<uint16_t*>(a.out) + (int64_t)(q.slot0 + c) * a.M + f;
          const int64_t pitch = C::kStaged ? 32 : a.M;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float v = __uint_as_float(z[i]);
            if (C::kStaged || i < left) store_bf16(out + i * pitch, v * gelu_gate(v));
          }
          if (C::kStaged) store_block(&a.mO, stage, blocks, q.m0 + lane0, q.slot0 + c);
        }
      } else if (MODE == FWD2 || MODE == DX) {
        const int f = q.m0 + lane0 + lane;
#pragma unroll 1
        for (int c = first; c < q.rows; c += step) {
          uint32_t z[32];
          ptx::tmem_ld_32x32b_x32(d + c, z);
          ptx::tmem_ld_wait();
          const int left = f < a.M ? q.rows - c : 0;
          // a token's largest finite value of these 32 columns is put into [2^14, 2^15); what is
          // above 2^-29 of it keeps fp16's precision.  The sum lifts a magnitude's exponent by one,
          // which makes infinities and NaN negative and so no maximum.
          const uint32_t magnitude = f < a.M ? 0x7fffffffu : 0u;
          int32_t mine = 0;  // lane i: the exponent of token c + i
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int32_t top = __reduce_max_sync(0xffffffffu, (int32_t)((z[i] & magnitude) + 0x00800000u));
            const int32_t e = max(top >> 23, 16);
            z[i] = __float_as_uint(__uint_as_float(z[i]) * __uint_as_float((uint32_t)(269 - e) << 23));
            if (lane == i) mine = e - 15;
          }
          uint16_t* out = C::kStaged ? stage_block(stage, blocks) + lane
                                     : reinterpret_cast<uint16_t*>(a.out) + (int64_t)(q.slot0 + c) * a.M + f;
          const int64_t pitch = C::kStaged ? 32 : a.M;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const __half2 h = __floats2half2_rn(__uint_as_float(z[i]), __uint_as_float(z[i + 1]));
            if (C::kStaged || i < left) out[i * pitch] = __half_as_ushort(__low2half(h));
            if (C::kStaged || i + 1 < left) out[(i + 1) * pitch] = __half_as_ushort(__high2half(h));
          }
          if (C::kStaged) store_block(&a.mO, stage, blocks, q.m0 + lane0, q.slot0 + c);
          if (c + lane < q.rows && q.m0 + lane0 < a.M)
            a.scale[scale_at(a.slots, q.slot0 + c + lane, (q.m0 + lane0) / 32)] = (uint8_t)mine;
        }
      } else if (C::kBwd1) {
        // The MMA's adder cuts what lies behind the accumulator's 24 bits, towards zero: normal
        // operands lose 1.2e-8 to 1.5e-8 of a sum in each step of 16 products (K = 256 to 8192), sums
        // that are exact nothing.  The values are taken as they are: no factor is right for both.
        const int f = q.m0 + lane0 + lane;
        const bool in = f < a.M;
#pragma unroll 1
        for (int c = first; c < q.rows; c += step) {
          const int nth = (c - first) / step;
          float dots[16];
          uint32_t z[16], u[16], g[16];
          ptx::tmem_ld_32x32b_x16(d + c, z);
          if (C::kG == 2) ptx::tmem_ld_32x32b_x16(d + C::kCols + c, u);
          ptx::tmem_ld_32x32b_x16(d + C::kG * C::kCols + c, g);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float w = __shfl_sync(0xffffffffu, w_held[0], nth % 2 * 16 + i);
            const float zz = __uint_as_float(z[i]), dh = __uint_as_float(g[i]), dhw = w * dh;
            float h, vz, vu = 0.0f;
            if (C::kG == 2) {
              const float uu = __uint_as_float(u[i]), sg = sigmoid_full(zz), zs = zz * sg;
              h = zs * uu;
              vz = dhw * uu * (sg + zs * (1.0f - sg));
              vu = dhw * zs;
            } else {
              const float sg = sigmoid_full(gelu_arg(zz));
              h = zz * sg;
              // far out, where the sigmoid is 0 or 1, the square must not become an infinity
              const float z2 = fminf(zz * zz, 1e30f);
              vz = dhw * (sg + h * (1.0f - sg) * 2.0f * kGeluC * (1.0f + 3.0f * 0.044715f * z2));
            }
            dots[i] = in ? dh * h : 0.0f;
            // two tokens to a register
            z[i] = __float_as_uint(vz);
            g[i] = __float_as_uint(w * h);
            if (C::kG == 2) u[i] = __float_as_uint(vu);
            if (i & 1) {
              z[i / 2] = pack2(__uint_as_float(z[i - 1]), __uint_as_float(z[i]));
              g[i / 2] = pack2(__uint_as_float(g[i - 1]), __uint_as_float(g[i]));
              if (C::kG == 2) u[i / 2] = pack2(__uint_as_float(u[i - 1]), __uint_as_float(u[i]));
            }
          }
          if (c + 16 > q.rows) {  // zeros behind the last row, to the end of these kRowStep
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int left = q.rows - c - 2 * i;
              const uint32_t kept = left <= 0 ? 0u : left == 1 ? 0xffffu : 0xffffffffu;
              z[i] &= kept;
              g[i] &= kept;
              if (C::kG == 2) u[i] &= kept;
            }
          }
          auto put = [&](const uint32_t (&v)[16], const CUtensorMap* m, int part) {
            if (lane == 0) ptx::bulk_wait_group_read<0>();
            __syncwarp();
            uint16_t* o = reinterpret_cast<uint16_t*>(stage) + lane;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[64 * i] = (uint16_t)v[i];
              o[64 * i + 32] = (uint16_t)(v[i] >> 16);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              ptx::tma_store_3d(m, stage, q.m0 + lane0, part, q.slot0 + c);
              ptx::bulk_commit_group();
            }
          };
          if (q.m0 + lane0 < a.M) {
            put(z, &a.mO, 0);
            if (C::kG == 2) put(u, &a.mO, 1);
            put(g, &a.mO2, 0);
          }
          const float s = transpose_sum(dots, lane);
          if (lane < 16 && c + lane < q.rows)
            a.part[(int64_t)(q.slot0 + c + lane) * a.parts + (q.m0 + lane0) / 32] = s;
          if (nth % 2) w_held[0] = w_held[1];
        }
      } else {
        // A lane holds 32 columns of its row: four 16-byte pieces of 64-byte rows, placed as the
        // map's 64-byte swizzle has them; rows and columns outside the matrix are not written.  Without the
        // stores the 4096-token case takes 59 us less, with every expert's operands in the L2 25.
        const bool second = q.e >= a.E;
        const CUtensorMap* mo = second ? &a.mO2 : &a.mO;
        const int rows = second ? a.M2 : a.M, width = second ? a.N2 : a.N, e = second ? q.e - a.E : q.e;
#pragma unroll 1
        for (int c = first; c < C::kCols; c += step) {
          uint32_t z[32];
          if (empty_tile) {
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] = 0;
          } else {
            ptx::tmem_ld_32x32b_x32(d + c, z);
            ptx::tmem_ld_wait();
          }
          if (q.n0 + c >= width || q.m0 + lane0 >= rows) continue;
          uint8_t* row = reinterpret_cast<uint8_t*>(stage_block(stage, blocks)) + lane * 64;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              p[j] = pack2(__uint_as_float(z[8 * i + 2 * j]), __uint_as_float(z[8 * i + 2 * j + 1]));
            *reinterpret_cast<uint4*>(row + ((i ^ (lane / 2)) & 3) * 16) = make_uint4(p[0], p[1], p[2], p[3]);
          }
          store_block(mo, stage, blocks, q.n0 + c, q.m0 + lane0, e);
        }
      }
      if (!empty_tile) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&tempty[buf]);
      }
    }
    if (C::kWarpOut && lane == 0) ptx::bulk_wait_group_all();  // the stores still read this warp's blocks
    if (!ok && lane == 0) {
      abort_flag = 1;
      a.plan[PLAN_ERR] = (int32_t)kErrWait;
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
