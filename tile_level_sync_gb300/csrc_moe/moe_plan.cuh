// The dispatch plan: a stable counting sort of the T * top_k expert ids.
//
// A plan is an array of 32-bit words: a header, the experts' counts, the offsets of their
// first slots (multiples of kTileRows, so that a 128-row tile of a product belongs to one
// expert), the row tiles {expert, first slot, rows} of up to 128, 160 and 256 rows, slot_of (assignment -> slot) and row_of (slot
// -> assignment).
//
// Blocks take consecutive chunks of the ids, a block's warps consecutive parts of its
// chunk.  Within 32 ids, equal ones find each other with one match instruction; the rank
// of an assignment is then the sum of what earlier blocks, warps and groups of 32 hold of
// its expert.  Nothing depends on the order in which blocks run.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "moe_ptx.cuh"

namespace cusync {
namespace moe {

constexpr int kTileRows = 128;
constexpr int kMidRows = 160;  // rows of BWD1's tiles on pairs
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kHeld = 4;  // groups of 32 ids whose ranks a warp keeps in registers
enum : int { PLAN_ERR = 0, PLAN_TILES = 2, PLAN_PAIRS = 3, PLAN_MIDS = 4, PLAN_COUNTERS = 8, PLAN_HEADER = 16 };

struct PlanArgs {
  const int32_t* ids;
  int32_t* plan;
  int64_t A;            // assignments
  int64_t S;            // slots
  int32_t E;
  int32_t blocks;       // 1: no histogram kernel ran
  int64_t chunk;        // assignments of a block (a multiple of kPlanThreads)
  int64_t counts, offsets, tiles, pairs, mids, slot_of, row_of, hist;  // word offsets
};

__device__ __forceinline__ int plan_id(const PlanArgs& a, int64_t i, int64_t end) {
  if (i >= end) return -1;
  const int id = a.ids[i];
  return (unsigned)id < (unsigned)a.E ? id : -1;
}

// Ids of each expert in every block's chunk: hist[block][expert].
__global__ void __launch_bounds__(kPlanThreads) plan_hist_kernel(PlanArgs a) {
  extern __shared__ uint32_t sh[];
  for (int e = threadIdx.x; e < a.E; e += kPlanThreads) sh[e] = 0;
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * a.chunk, end = min(a.A, lo + a.chunk);
  for (int64_t i = lo + threadIdx.x; i < end; i += kPlanThreads) {
    const int id = plan_id(a, i, end);
    if (id >= 0) atomicAdd(&sh[id], 1u);
  }
  __syncthreads();
  uint32_t* h = reinterpret_cast<uint32_t*>(a.plan + a.hist) + (int64_t)blockIdx.x * a.E;
  for (int e = threadIdx.x; e < a.E; e += kPlanThreads) h[e] = sh[e];
}

// An expert's c rows from slot o on, as tiles {expert, first slot, rows} of `most` rows and
// one of the rest: a product's time goes by the bytes it loads, which a full tile uses best.
__device__ __forceinline__ void cut_tiles(int4* out, int e, int o, int c, int most, int lane) {
  for (int i = lane; i * most < c; i += 32) out[i] = make_int4(e, o + i * most, min(most, c - i * most), 0);
}

// Shared memory of plan_kernel: per-warp histograms [kPlanWarps][E], then before[E],
// count[E], offset[E + 1], pair[E + 1], mid[E + 1], and the scan's 32 partial sums of 64 bits.
__host__ __device__ inline int plan_scan_at(int E) { return (kPlanWarps * E + 5 * E + 3 + 1) & ~1; }
__host__ __device__ inline size_t plan_smem(int E) { return (size_t)plan_scan_at(E) * 4 + 32 * 8; }

__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(PlanArgs a) {
  extern __shared__ uint32_t sh[];
  const int E = a.E, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* whist = sh;
  uint32_t* before = whist + kPlanWarps * E;
  uint32_t* count = before + E;
  uint32_t* offset = count + E;
  uint32_t* pair = offset + E + 1;
  uint32_t* mid = pair + E + 1;
  uint64_t* part = reinterpret_cast<uint64_t*>(sh + plan_scan_at(E));
  for (int i = tid; i < kPlanWarps * E; i += kPlanThreads) whist[i] = 0;
  for (int e = tid; e < E; e += kPlanThreads) before[e] = count[e] = 0;
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  __syncthreads();

  // this warp's part of the chunk: ranks within the warp, the first kHeld groups' in
  // registers, what comes behind them in slot_of for now
  const int64_t lo = (int64_t)blockIdx.x * a.chunk, end = min(a.A, lo + a.chunk);
  const int64_t per_warp = a.chunk / kPlanWarps;
  const int64_t w0 = lo + warp * per_warp, w1 = min(end, w0 + per_warp);
  uint32_t* mine = whist + warp * E;
  int32_t* slot_of = a.plan + a.slot_of;
  auto rank_of = [&](int id) {
    const unsigned same = __match_any_sync(0xffffffffu, id), lower = same & ((1u << lane) - 1);
    const uint32_t seen = id >= 0 ? mine[id] : 0;
    __syncwarp();
    if (id >= 0 && lower == 0) mine[id] = seen + __popc(same);
    __syncwarp();
    return seen + __popc(lower);
  };
  int held_id[kHeld];
  uint32_t held[kHeld];
#pragma unroll
  for (int h = 0; h < kHeld; ++h) held_id[h] = plan_id(a, w0 + 32 * h + lane, w1);
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
    if (w0 + 32 * h < w1) held[h] = rank_of(held_id[h]);
  for (int64_t i0 = w0 + 32 * kHeld; i0 < w1; i0 += 32) {
    const uint32_t r = rank_of(plan_id(a, i0 + lane, w1));
    if (i0 + lane < w1) slot_of[i0 + lane] = (int32_t)r;
  }
  // what other blocks hold: all of it into count, the earlier blocks' into before
  if (a.blocks > 1) {
    const uint32_t* h = reinterpret_cast<const uint32_t*>(a.plan + a.hist);
    const int rows = kPlanThreads / E;  // block rows summed side by side (E <= kPlanThreads)
    const int e = tid % E, r = tid / E;
    if (r < rows) {
      uint32_t all = 0, early = 0;
#pragma unroll 8
      for (int b = r; b < a.blocks; b += rows) {
        const uint32_t v = __ldcg(h + (int64_t)b * E + e);
        all += v;
        if (b < (int)blockIdx.x) early += v;
      }
      atomicAdd(&count[e], all);  // whole numbers: any order
      atomicAdd(&before[e], early);
    }
  }
  __syncthreads();
  // exclusive prefix over the warps; one block alone has the counts now
  for (int e = tid; e < E; e += kPlanThreads) {
    uint32_t c = 0;
#pragma unroll 8
    for (int w = 0; w < kPlanWarps; ++w) {
      const uint32_t v = whist[w * E + e];
      whist[w * E + e] = c;
      c += v;
    }
    if (a.blocks == 1) count[e] = c;
  }
  __syncthreads();
  // offsets: exclusive scans of the counts in whole tiles of each kind (E <= kPlanThreads)
  {
    const uint32_t n = tid < E ? count[tid] : 0;
    // 21 bits each (at most 2^17 + 2^10 tiles): of 128 rows, of 256, of 160
    const uint64_t v = (n + kTileRows - 1) / kTileRows + ((uint64_t)((n + 2 * kTileRows - 1) / (2 * kTileRows)) << 21) +
                       ((uint64_t)((n + kMidRows - 1) / kMidRows) << 42);
    uint64_t s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    if (lane == 31) part[warp] = s;
    __syncthreads();
    if (warp == 0) {
      const uint64_t p = part[lane];
      uint64_t q = p;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t u = __shfl_up_sync(0xffffffffu, q, o);
        if (lane >= o) q += u;
      }
      part[lane] = q - p;
    }
    __syncthreads();
    if (tid < E) {
      s += part[warp];
      const uint64_t from = s - v;
      offset[tid] = (uint32_t)(from & 0x1fffff) * kTileRows;
      pair[tid] = (uint32_t)(from >> 21) & 0x1fffff;
      mid[tid] = (uint32_t)(from >> 42);
      if (tid == E - 1) {
        offset[E] = (uint32_t)(s & 0x1fffff) * kTileRows;
        pair[E] = (uint32_t)(s >> 21) & 0x1fffff;
        mid[E] = (uint32_t)(s >> 42);
      }
    }
  }
  __syncthreads();
  const int64_t used = offset[E];
  if (blockIdx.x == 0) {
    if (tid < PLAN_HEADER - PLAN_COUNTERS) a.plan[PLAN_COUNTERS + tid] = 0;  // tiles claimed by each product
    if (tid == 0) {
      a.plan[PLAN_ERR] = 0;
      a.plan[PLAN_TILES] = (int32_t)(used / kTileRows);
      a.plan[PLAN_PAIRS] = (int32_t)pair[E];
      a.plan[PLAN_MIDS] = (int32_t)mid[E];
    }
    for (int e = tid; e < E; e += kPlanThreads) a.plan[a.counts + e] = (int32_t)count[e];
    for (int e = tid; e <= E; e += kPlanThreads) a.plan[a.offsets + e] = (int32_t)offset[e];
  }
  // an expert's tiles and the slots behind its last row: the experts shared among blocks
  int32_t* row_of = a.plan + a.row_of;
  for (int e = blockIdx.x * kPlanWarps + warp; e < E; e += gridDim.x * kPlanWarps) {
    const int64_t o = offset[e], n = offset[e + 1];
    const int c = (int)count[e];
    cut_tiles(reinterpret_cast<int4*>(a.plan + a.tiles) + o / kTileRows, e, (int)o, c, kTileRows, lane);
    cut_tiles(reinterpret_cast<int4*>(a.plan + a.pairs) + pair[e], e, (int)o, c, 2 * kTileRows, lane);
    cut_tiles(reinterpret_cast<int4*>(a.plan + a.mids) + mid[e], e, (int)o, c, kMidRows, lane);
    for (int64_t i = o + count[e] + lane; i < n; i += 32) row_of[i] = -1;
  }
  for (int64_t i = used + (int64_t)blockIdx.x * kPlanThreads + tid; i < a.S; i += (int64_t)gridDim.x * kPlanThreads)
    row_of[i] = -1;
  auto place = [&](int64_t i, int id, uint32_t rank) {
    const uint32_t s = id >= 0 ? offset[id] + before[id] + mine[id] + rank : 0xffffffffu;
    slot_of[i] = (int32_t)s;  // -1: no expert
    if (id >= 0) row_of[s] = (int32_t)i;
  };
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
    if (w0 + 32 * h + lane < w1) place(w0 + 32 * h + lane, held_id[h], held[h]);
  for (int64_t i = w0 + 32 * kHeld + lane; i < w1; i += 32) place(i, plan_id(a, i, w1), (uint32_t)slot_of[i]);
}

}  // namespace moe
}  // namespace cusync
