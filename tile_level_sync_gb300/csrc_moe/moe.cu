// Host side of include/cusync_moe.h: argument checks, buffer layouts, TMA descriptors and
// kernel launches of the expert layer.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include "../../include/cusync_moe.h"
#include "moe_gemm.cuh"
#include "moe_launch.h"
#include "moe_plan.cuh"
#include "moe_small.cuh"

using namespace cusync;
using namespace cusync::moe;

namespace {

static_assert(kTileRows == CUSYNC_MOE_TILE_ROWS, "the plan's alignment");
static_assert(CUSYNC_MOE_MAX_EXPERTS <= kPlanThreads, "the plan scans the experts in one step");

constexpr int64_t kPlanAlone = 2048;   // assignments that one plan block takes
constexpr int64_t kPlanChunk = 1024;   // assignments of a plan block, where there are more
constexpr int64_t kPlanBlocks = 64;    // plan blocks at most
// Assignments up to which the MLP runs without tiles.  It reads an expert's weights once for each
// assignment, which is right where a call's tokens choose different experts (us, without and with
// tiles; 64 experts, 8 a token, D 2048, N1 1024: 1 token 22.7 / 35.2, 2 40.9 / 51.9, 4 69.7 / 71.8).
// Where they share experts, or one assignment's weights are large, tiles are faster below the
// border already, which goes by the count alone (8 experts, 2 a token: 1 token 13.3 / 24.2,
// 4 31.5 / 27.3, 16 88.9 / 32.9; with D 4096, N1 14336 1 token 180 / 133, 16 2545 / 430).
constexpr int64_t kSmallAssignments = 32;
// Assignments per expert from which products take tiles of 256 rows on pairs of CTAs (us of the
// MLP, single CTAs / pairs; 64 experts, 8 a token, D 2048, N1 1024: 64 an expert 162.8 / 166.2,
// 96 169.9 / 172.9, 128 187.0 / 181.6, 192 231.4 / 199.5, 256 265.8 / 230.9).
constexpr int64_t kPairRows = 128;
// Assignments per expert up to which the first product gathers the tokens' rows itself (the same
// layer, copied / gathered: 8 an expert 145.1 / 141.1, 16 147.6 / 144.2, 24 151.7 / 150.8,
// 32 154.3 / 157.2).
constexpr int64_t kGatherRows = 16;

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return div_up(a, b) * b; }
bool aligned(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// What a descriptor means, its defaults filled in.
struct Layer {
  int64_t T, D, N1, A, S, max_pairs, max_mids;
  int32_t E, k, G, groups, group_limit, group_top;
  int64_t chunk, blocks;                                          // plan
  int64_t counts, offsets, tiles, pairs, mids, slot_of, row_of, hist;  // plan, 32-bit words
  int64_t plan_bytes;
  int64_t x, h, rows, scales, work_bytes;                                // forward work, bytes
  int64_t gx, gy, gh, gz, grows, gscales, gpart, grad_bytes;                      // gradient work, bytes
  int32_t parts;
};

cusync_status_t read_desc(const cusync_moe_desc_t* d, Layer* L, bool mlp) {
  if (!d) return CUSYNC_ERR_INVALID_ARG;
  if (d->T < 0 || d->experts < 1 || d->top_k < 1 || d->groups < 0 || d->group_limit < 0 || d->num_sms < 0 ||
      d->D < 0 || d->N1 < 0)
    return CUSYNC_ERR_INVALID_ARG;
  if ((d->act != CUSYNC_MOE_GELU && d->act != CUSYNC_MOE_SWIGLU) ||
      (d->score != CUSYNC_MOE_SOFTMAX && d->score != CUSYNC_MOE_SIGMOID) || d->group_top < 0 || d->group_top > 2 ||
      !std::isfinite(d->scale))
    return CUSYNC_ERR_INVALID_ARG;
  L->groups = d->groups ? d->groups : 1;
  L->group_limit = d->group_limit ? d->group_limit : L->groups;
  L->group_top = d->group_top ? d->group_top : 1;
  if (d->experts > CUSYNC_MOE_MAX_EXPERTS || d->top_k > CUSYNC_MOE_MAX_TOP_K || L->groups > CUSYNC_MOE_MAX_GROUPS)
    return CUSYNC_ERR_UNSUPPORTED;
  if (d->experts % L->groups || L->group_limit > L->groups ||
      d->top_k > L->group_limit * (d->experts / L->groups))
    return CUSYNC_ERR_INVALID_ARG;
  if (d->T > CUSYNC_MOE_MAX_ASSIGNMENTS / d->top_k) return CUSYNC_ERR_UNSUPPORTED;
  if (mlp) {
    if (d->D < 1 || d->N1 < 1) return CUSYNC_ERR_INVALID_ARG;
    if (d->D % 8 || d->N1 % 8 || d->D > (1 << 20) || d->N1 > (1 << 20)) return CUSYNC_ERR_UNSUPPORTED;
    // the kernels count weight rows and tiles in 32 bits
    const int64_t rows = (int64_t)d->experts * std::max(2 * d->N1, d->D);
    const int64_t row_tiles = d->T * d->top_k / kTileRows + d->experts;
    const int64_t tiles = std::max(row_tiles * div_up(std::max(d->N1, d->D), 64),
                                   d->experts * div_up(2 * d->N1, 128) * div_up(d->D, 128));
    if (rows > INT32_MAX || tiles > INT32_MAX / 2) return CUSYNC_ERR_UNSUPPORTED;
  }
  L->T = d->T;
  L->D = d->D;
  L->N1 = d->N1;
  L->E = d->experts;
  L->k = d->top_k;
  L->G = d->act == CUSYNC_MOE_SWIGLU ? 2 : 1;
  L->A = L->T * L->k;
  L->S = round_up(L->A + (kTileRows - 1) * std::min<int64_t>(L->E, L->A), kTileRows);
  L->chunk = L->A <= kPlanAlone ? kPlanAlone : std::max(kPlanChunk, round_up(div_up(L->A, kPlanBlocks), kPlanThreads));
  L->blocks = std::max<int64_t>(1, div_up(L->A, L->chunk));
  int64_t w = PLAN_HEADER;
  auto take = [&w](int64_t n) {
    const int64_t at = w;
    w += round_up(n, 4);
    return at;
  };
  L->counts = take(L->E);
  L->offsets = take(L->E + 1);
  L->tiles = take(4 * (L->S / kTileRows));
  L->max_pairs = L->A / (2 * kTileRows) + std::min<int64_t>(L->E, L->A);
  L->pairs = take(4 * L->max_pairs);
  L->max_mids = L->A / kMidRows + std::min<int64_t>(L->E, L->A);
  L->mids = take(4 * L->max_mids);
  L->slot_of = take(L->A);
  L->row_of = take(L->S);
  L->hist = take(L->blocks > 1 ? L->blocks * L->E : 0);
  L->plan_bytes = round_up(w * 4, 256);
  L->x = L->h = L->rows = L->scales = L->gscales = L->work_bytes = L->gx = L->gy = L->gh = L->gz = L->grows = L->gpart = L->grad_bytes = 0;
  L->parts = 0;
  if (d->D >= 1 && d->N1 >= 1) {
    int64_t b = L->plan_bytes;
    auto bytes = [&b](int64_t n) {
      const int64_t at = b;
      b += round_up(n, 256);
      return at;
    };
    L->x = bytes(L->S * L->D * 2);
    L->h = bytes(L->S * L->N1 * 2);
    L->rows = bytes(L->S * L->D * 2);
    L->scales = bytes(L->S * 8 * div_up(L->D, 256));
    L->work_bytes = b;
    b = L->plan_bytes;
    L->parts = (int32_t)(8 * div_up(L->N1, 256));  // one for 32 columns
    L->gx = bytes(L->S * L->D * 2);
    L->gy = bytes(L->S * L->D * 2);
    L->gh = bytes(L->S * L->N1 * 2);
    L->gz = bytes(L->S * L->G * L->N1 * 2);
    L->grows = bytes(L->S * L->D * 2);
    L->gscales = bytes(L->S * 8 * div_up(L->D, 256));
    L->gpart = bytes(L->S * L->parts * 4);
    L->grad_bytes = b;
  }
  return CUSYNC_OK;
}

// ----------------------------------------------------------------------------- devices

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::mutex g_mu;
constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];  // SMs of a prepared device, 0 = not prepared

template <int MODE, int ACT, int PAIR>
cudaError_t prepare_gemm() {
  const void* f = reinterpret_cast<const void*>(&moe_gemm_kernel<MODE, ACT, PAIR>);
  cudaError_t e =
      cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, GemmCfg<MODE, ACT, PAIR>::kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;  // loads the kernel now, not at a launch inside a capture
  return cudaFuncGetAttributes(&fa, f);
}

template <int PAIR>
cudaError_t prepare_pair() {
  cudaError_t e = prepare_gemm<FWD1, 0, PAIR>();
  if (e == cudaSuccess) e = prepare_gemm<FWD1, 1, PAIR>();
  if (e == cudaSuccess) e = prepare_gemm<FWD2, 0, PAIR>();
  if (e == cudaSuccess) e = prepare_gemm<BWD1, 0, PAIR>();
  if (e == cudaSuccess) e = prepare_gemm<BWD1, 1, PAIR>();
  if (e == cudaSuccess) e = prepare_gemm<DX, 0, PAIR>();
  if (e == cudaSuccess) e = prepare_gemm<DW, 0, PAIR>();
  return e;
}

// The current device: the attributes set of the kernels that need some, the descriptor encoder
// found.  The first call on a device does the work.  The kernels without attributes (router,
// copies, sums, few tokens) are loaded by their first launch.
cusync_status_t prepare_device(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) return CUSYNC_ERR_CUDA;
  if (int n = g_sms[dev].load(std::memory_order_acquire)) {
    *sms = n;
    return CUSYNC_OK;
  }
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn)
      return CUSYNC_ERR_CUDA;
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  int n = 0;
  cudaError_t e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = prepare_pair<1>();
  if (e == cudaSuccess) e = prepare_pair<2>();
  if (e == cudaSuccess) e = prepare_gemm<FWD1G, 0, 1>();
  if (e == cudaSuccess) e = prepare_gemm<FWD1G, 1, 1>();
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)plan_smem(CUSYNC_MOE_MAX_EXPERTS));
  if (e != cudaSuccess) return CUSYNC_ERR_CUDA;
  g_sms[dev].store(n, std::memory_order_release);
  *sms = n;
  return CUSYNC_OK;
}

// A map of bf16 elements: sizes and strides (in elements, from the second dimension on) and
// the box, innermost first; 128-byte swizzle; elements outside read as zero.
template <int N>
bool map_nd(CUtensorMap* m, const void* p, const int64_t (&size)[N], const int64_t (&stride)[N - 1],
            const int (&box_size)[N]) {
  cuuint64_t dims[N], strides[N - 1];
  cuuint32_t box[N], one[N];
  for (int i = 0; i < N; ++i) {
    dims[i] = (cuuint64_t)size[i];
    box[i] = (cuuint32_t)box_size[i];
    one[i] = 1;
    if (i) strides[i - 1] = (cuuint64_t)stride[i - 1] * 2;
  }
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, N, const_cast<void*>(p), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows [rows, cols]: boxes of 64 columns x box_rows; wide: [cols / 64][rows][64], boxes of
// `chunks` times that.
bool map_rows(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int box_rows, bool wide, int chunks) {
  return wide ? map_nd<3>(m, p, {64, rows, cols / 64}, {cols, 64}, {64, box_rows, chunks})
              : map_nd<2>(m, p, {cols, rows}, {cols}, {64, box_rows});
}
// Matrices [depth][rows, cols], the depth a dimension of its own (rows outside a matrix read
// as zero); wide: their rows one after the other, as above.
bool map_weights(CUtensorMap* m, const void* p, int64_t depth, int64_t rows, int64_t cols, int box_rows, bool wide,
                 int chunks) {
  return wide ? map_rows(m, p, depth * rows, cols, box_rows, true, chunks)
              : map_nd<3>(m, p, {cols, rows, depth}, {cols, rows * cols}, {64, box_rows, 1});
}
// W1t of a gated layer with gate and up rows eight by eight, 64 of each at a time: the rows
// as [N1/8 of every expert][2][8].  wide: all experts' rows as one run of eights, which ends
// N1 early so that the up rows of the last one stay inside.
bool map_gated(CUtensorMap* m, const void* p, int64_t experts, int64_t n1, int64_t d, bool wide, int blocks) {
  return wide ? map_nd<5>(m, p, {64, 8, 2, (2 * experts - 1) * n1 / 8, d / 64}, {d, n1 * d, 8 * d, 64},
                          {64, 8, 2, 8, blocks})
              : map_nd<5>(m, p, {d, 8, 2, n1 / 8, experts}, {d, n1 * d, 8 * d, 2 * n1 * d}, {64, 8, 2, 8, 1});
}
// W1t's rows for BWD1: 128 gate and the 128 up rows N1 further (GeLU: 128 rows).
bool map_gate_up(CUtensorMap* m, const void* p, int64_t experts, int g, int64_t n1, int64_t d, bool wide) {
  if (!wide) return map_weights(m, p, experts * g, n1, d, 128, false, 1);
  return map_nd<3>(m, p, {d, (g * experts - (g - 1)) * n1, g}, {d, n1 * d}, {64, 128, g});
}
// An output by slot: boxes of `cols` columns (a warp's) x 32 rows as they lie in shared memory.
bool map_output(CUtensorMap* m, const void* p, int64_t rows, int64_t width, int cols) {
  cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)width * 2};
  cuuint32_t box[2] = {(cuuint32_t)cols, 32}, one[2] = {1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(p), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// A weight gradient [experts][rows, cols]: boxes of 32 x 32, 64-byte swizzle.
bool map_gradient(CUtensorMap* m, void* p, int64_t experts, int64_t rows, int64_t cols) {
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)experts};
  cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)(rows * cols) * 2};
  cuuint32_t box[3] = {32, 32, 1}, one[3] = {1, 1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// dZ or w H by slot, [slots][g, cols]: boxes of 16 slots x 32 columns of one of the g parts.
bool map_hidden(CUtensorMap* m, void* p, int64_t slots, int64_t g, int64_t cols) {
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)g, (cuuint64_t)slots};
  cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)(g * cols) * 2};
  cuuint32_t box[3] = {32, 1, 16}, one[3] = {1, 1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Token rows by slot, in the four box heights.
bool map_tokens(CUtensorMap (&m)[4], const void* p, int64_t rows, int64_t cols, bool wide, int blocks, int last = 128) {
  bool ok = true;
  for (int i = 0; i < 4; ++i) ok = ok && map_rows(&m[i], p, rows, cols, i < 3 ? 16 << i : last, wide, blocks);
  return ok;
}

// ----------------------------------------------------------------------------- launches

template <bool GRAD>
cusync_status_t route_any(const cusync_moe_desc_t* d, const Layer& L, RouteArgs a, cudaStream_t s) {
  a.T = L.T;
  a.E = L.E;
  a.k = L.k;
  a.groups = L.groups;
  a.group_size = L.E / L.groups;
  a.group_limit = L.group_limit;
  a.group_top = L.group_top;
  a.renorm = d->renorm ? 1 : 0;
  a.scale = d->scale;
  if (L.T == 0) return CUSYNC_OK;
  int sms = 0;
  const cusync_status_t st = prepare_device(&sms);
  if (st != CUSYNC_OK) return st;
  if (d->num_sms) sms = std::min(sms, d->num_sms);
  const bool soft = d->score == CUSYNC_MOE_SOFTMAX;
  const cudaError_t e = d->logits_f32 ? route_f32(a, soft, GRAD, sms, s) : route_bf16(a, soft, GRAD, sms, s);
  return e == cudaSuccess ? CUSYNC_OK : CUSYNC_ERR_CUDA;
}

cudaError_t launch_plan(const Layer& L, const int32_t* ids, void* plan, cudaStream_t s) {
  PlanArgs p = {};
  p.ids = ids;
  p.plan = static_cast<int32_t*>(plan);
  p.A = L.A;
  p.S = L.S;
  p.E = L.E;
  p.blocks = (int32_t)L.blocks;
  p.chunk = L.chunk;
  p.counts = L.counts;
  p.offsets = L.offsets;
  p.tiles = L.tiles;
  p.pairs = L.pairs;
  p.mids = L.mids;
  p.slot_of = L.slot_of;
  p.row_of = L.row_of;
  p.hist = L.hist;
  if (L.blocks > 1) {
    const cudaError_t e = launch(plan_hist_kernel, dim3((unsigned)L.blocks), kPlanThreads, (size_t)L.E * 4, s, p);
    if (e != cudaSuccess) return e;
  }
  return launch(plan_kernel, dim3((unsigned)L.blocks), kPlanThreads, plan_smem(L.E), s, p);
}

GemmArgs gemm_args(const Layer& L, void* work, const float* weights) {
  GemmArgs a;
  std::memset(&a, 0, sizeof(a));
  a.plan = static_cast<int32_t*>(work);
  a.weights = weights;
  a.counts = L.counts;
  a.offsets = L.offsets;
  a.tiles = L.tiles;
  a.row_of = L.row_of;
  a.T = (int32_t)L.T;
  a.k = L.k;
  a.E = L.E;
  a.slots = (int32_t)L.S;
  return a;
}

template <int MODE, int ACT, int PAIR>
cudaError_t launch_gemm(GemmArgs a, const Layer& L, int sms, cudaStream_t s) {
  static_assert(MODE <= DW || MODE == FWD1G, "one counter for each product of a call");
  a.counter = PLAN_COUNTERS + (MODE == FWD1G ? FWD1 : MODE);
  using C = GemmCfg<MODE, ACT, PAIR>;
  constexpr int count = C::kTileCount;
  a.tiles = count == PLAN_PAIRS ? L.pairs : count == PLAN_MIDS ? L.mids : L.tiles;
  const int64_t row_tiles = count == PLAN_PAIRS ? L.max_pairs : count == PLAN_MIDS ? L.max_mids : L.S / kTileRows;
  a.m_tiles = (int32_t)div_up(a.M, C::kFeatures);
  a.n_tiles = C::kDw ? (int32_t)div_up(a.N, C::kCols) : 1;
  a.m_tiles2 = (int32_t)div_up(a.M2, C::kFeatures);  // DW
  a.n_tiles2 = (int32_t)div_up(a.N2, C::kCols);
  // an upper bound: how many tiles of rows there are is only known on the device
  const int64_t tiles = C::kDw ? a.E * ((int64_t)a.m_tiles * a.n_tiles + (int64_t)a.m_tiles2 * a.n_tiles2)
                               : row_tiles * a.m_tiles;
  const int grid = PAIR * (int)std::max<int64_t>(1, std::min<int64_t>(tiles, sms / PAIR));
  return launch_cluster(PAIR, moe_gemm_kernel<MODE, ACT, PAIR>, dim3(grid), C::kThreads, C::kSmemBytes, s, a);
}
template <int MODE, int ACT>
cudaError_t launch_gemm(bool pair, const GemmArgs& a, const Layer& L, int sms, cudaStream_t s) {
  return pair ? launch_gemm<MODE, ACT, 2>(a, L, sms, s) : launch_gemm<MODE, ACT, 1>(a, L, sms, s);
}

bool use_pairs(const Layer& L, int sms) { return L.A >= kPairRows * L.E && sms >= 2; }

cudaError_t launch_dispatch(const Layer& L, void* work, const void* x, void* xs, const void* y, void* ys, cudaStream_t s) {
  DispatchArgs d = {};
  d.plan = static_cast<int32_t*>(work);
  d.x = static_cast<const uint4*>(x);
  d.xs = static_cast<uint4*>(xs);
  d.y = static_cast<const uint4*>(y);
  d.ys = static_cast<uint4*>(ys);
  d.T = L.T;
  d.slot_of = L.slot_of;
  d.counts = L.counts;
  d.offsets = L.offsets;
  d.k = (int32_t)L.k;
  d.E = (int32_t)L.E;
  d.chunks = (int32_t)(L.D / 8);
  const int64_t blocks = div_up((L.T + L.E) * d.chunks, kDispatchThreads);  // 2^31 of them would be an X of 8 TB
  return launch(dispatch_kernel, dim3((unsigned)blocks), kDispatchThreads, 0, s, d);
}

cudaError_t launch_combine(const Layer& L, void* work, const void* rows, const void* scale, const float* weights,
                           void* out, const float* part, float* dweights, cudaStream_t s) {
  CombineArgs c = {};
  c.plan = static_cast<int32_t*>(work);
  c.rows = static_cast<const __half*>(rows);
  c.scale = static_cast<const uint8_t*>(scale);
  c.slots = (int32_t)L.S;
  c.weights = weights;
  c.out = out;
  c.part = part;
  c.dweights = dweights;
  c.slot_of = L.slot_of;
  c.T = (int32_t)L.T;
  c.k = L.k;
  c.D = (int32_t)L.D;
  c.parts = L.parts;
  c.used = (int32_t)div_up(L.N1, 32);
  return launch(combine_kernel, dim3((unsigned)L.T, (unsigned)div_up(L.D, 8 * kCombineThreads)), kCombineThreads, 0, s,
                c);
}

cusync_status_t status_of(cudaError_t e) { return e == cudaSuccess ? CUSYNC_OK : CUSYNC_ERR_CUDA; }

// The error word of a buffer that no kernel of the call touches (no token; work may be null).
cudaError_t clear_error(void* work, cudaStream_t s) {
  return aligned(work) ? cudaMemsetAsync(static_cast<int32_t*>(work) + PLAN_ERR, 0, 4, s) : cudaSuccess;
}

}  // namespace

extern "C" {

cusync_status_t cusync_moe_info(const cusync_moe_desc_t* d, cusync_moe_info_t* out) {
  Layer L;
  if (!out) return CUSYNC_ERR_INVALID_ARG;
  const bool mlp = d && (d->D != 0 || d->N1 != 0);
  const cusync_status_t st = read_desc(d, &L, mlp);
  if (st != CUSYNC_OK) return st;
  out->plan_bytes = L.plan_bytes;
  out->work_bytes = L.work_bytes;
  out->grad_work_bytes = L.grad_bytes;
  out->slots = L.S;
  out->counts = L.counts;
  out->offsets = L.offsets;
  out->slot_of = L.slot_of;
  out->row_of = L.row_of;
  return CUSYNC_OK;
}

cusync_status_t cusync_moe_route(const cusync_moe_desc_t* d, const void* logits, const float* bias, int32_t* ids,
                                 float* weights, cusync_stream_t stream) {
  Layer L;
  const cusync_status_t st = read_desc(d, &L, false);
  if (st != CUSYNC_OK) return st;
  if (L.T && (!aligned(logits) || !aligned(ids) || !aligned(weights) || (bias && !aligned(bias))))
    return CUSYNC_ERR_INVALID_ARG;
  RouteArgs a = {};
  a.logits = logits;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  return route_any<false>(d, L, a, (cudaStream_t)stream);
}

cusync_status_t cusync_moe_route_grad(const cusync_moe_desc_t* d, const void* logits, const int32_t* ids,
                                      const float* dweights, void* dlogits, cusync_stream_t stream) {
  Layer L;
  const cusync_status_t st = read_desc(d, &L, false);
  if (st != CUSYNC_OK) return st;
  if (L.T && (!aligned(logits) || !aligned(ids) || !aligned(dweights) || !aligned(dlogits)))
    return CUSYNC_ERR_INVALID_ARG;
  RouteArgs a = {};
  a.logits = logits;
  a.ids = const_cast<int32_t*>(ids);
  a.weights = const_cast<float*>(dweights);
  a.dlogits = dlogits;
  return route_any<true>(d, L, a, (cudaStream_t)stream);
}

cusync_status_t cusync_moe_plan(const cusync_moe_desc_t* d, const int32_t* ids, void* plan, cusync_stream_t stream) {
  Layer L;
  cusync_status_t st = read_desc(d, &L, false);
  if (st != CUSYNC_OK) return st;
  if ((L.A && !aligned(ids)) || !aligned(plan)) return CUSYNC_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = prepare_device(&sms)) != CUSYNC_OK) return st;
  return status_of(launch_plan(L, ids, plan, (cudaStream_t)stream));
}

cusync_status_t cusync_moe_mlp(const cusync_moe_desc_t* d, const void* X, const void* W1t, const void* W2t,
                               const int32_t* ids, const float* weights, void* work, void* Y,
                               cusync_stream_t stream) {
  Layer L;
  cusync_status_t st = read_desc(d, &L, true);
  if (st != CUSYNC_OK) return st;
  if (L.T == 0) return status_of(clear_error(work, (cudaStream_t)stream));
  if (!aligned(X) || !aligned(W1t) || !aligned(W2t) || !aligned(ids) || !aligned(weights) || !aligned(work) ||
      !aligned(Y))
    return CUSYNC_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = prepare_device(&sms)) != CUSYNC_OK) return st;
  if (d->num_sms) sms = std::min(sms, d->num_sms);
  cudaStream_t s = (cudaStream_t)stream;
  char* w = static_cast<char*>(work);
  if (L.A <= kSmallAssignments) {
    SmallArgs a = {};
    a.X = static_cast<const uint16_t*>(X);
    a.W1t = static_cast<const uint16_t*>(W1t);
    a.W2t = static_cast<const uint16_t*>(W2t);
    a.ids = ids;
    a.weights = weights;
    a.h = reinterpret_cast<float*>(w + L.h);
    a.Y = static_cast<uint16_t*>(Y);
    a.err = static_cast<int32_t*>(work);
    a.T = (int32_t)L.T;
    a.k = L.k;
    a.E = L.E;
    a.D = (int32_t)L.D;
    a.N1 = (int32_t)L.N1;
    const int64_t most = (int64_t)sms * kSmallBlocks;
    const dim3 up((unsigned)std::min(most, div_up(L.A * L.N1, kSmallThreads / 32)));
    const dim3 down((unsigned)std::min(most, div_up(L.T * L.D, kDownUnits)));
    cudaError_t e = L.G == 2 ? launch(small_up_kernel<1>, up, kSmallThreads, 0, s, a)
                             : launch(small_up_kernel<0>, up, kSmallThreads, 0, s, a);
    if (e == cudaSuccess) e = launch(small_down_kernel, down, kSmallThreads, 0, s, a);
    return status_of(e);
  }
  cudaError_t e = launch_plan(L, ids, work, s);
  if (e != cudaSuccess) return CUSYNC_ERR_CUDA;
  const bool gather = L.A <= kGatherRows * L.E, pair = use_pairs(L, sms);
  GemmArgs a = gemm_args(L, work, weights);
  a.M = (int32_t)L.N1;
  a.K = (int32_t)L.D;
  a.out = w + L.h;
  GemmArgs b = gemm_args(L, work, weights);
  b.M = (int32_t)L.D;
  b.K = (int32_t)L.N1;
  b.out = w + L.rows;
  b.scale = reinterpret_cast<uint8_t*>(w + L.scales);
  const bool wide = L.D % 64 == 0 && L.N1 % 64 == 0;
  a.wide = b.wide = wide;
  if (!(L.G == 2 ? map_gated(&a.mA, W1t, L.E, L.N1, L.D, wide, 2)
                 : map_weights(&a.mA, W1t, L.E, L.N1, L.D, 128, wide, 2)) ||
      !(gather ? map_rows(&a.mB[0], X, L.T, L.D, 1, false, 1) : map_tokens(a.mB, w + L.x, L.S, L.D, wide, 2)) ||
      !map_weights(&b.mA, W2t, L.E, L.D, L.N1, 128, wide, 2) || !map_tokens(b.mB, w + L.h, L.S, L.N1, wide, 2) ||
      !map_output(&a.mO, w + L.h, L.S, L.N1, 32 / L.G) || !map_output(&b.mO, w + L.rows, L.S, L.D, 32))
    return CUSYNC_ERR_CUDA;
  if (gather) {
    for (int i = 1; i < 4; ++i) a.mB[i] = a.mB[0];
    e = L.G == 2 ? launch_gemm<FWD1G, 1, 1>(a, L, sms, s) : launch_gemm<FWD1G, 0, 1>(a, L, sms, s);
  } else {
    e = launch_dispatch(L, work, X, w + L.x, nullptr, nullptr, s);
    if (e == cudaSuccess)
      e = L.G == 2 ? launch_gemm<FWD1, 1>(pair, a, L, sms, s) : launch_gemm<FWD1, 0>(pair, a, L, sms, s);
  }
  if (e == cudaSuccess) e = launch_gemm<FWD2, 0>(pair, b, L, sms, s);
  if (e == cudaSuccess)
    e = launch_combine(L, work, w + L.rows, w + L.scales, weights, Y, nullptr, nullptr, s);
  return status_of(e);
}

cusync_status_t cusync_moe_mlp_grad(const cusync_moe_desc_t* d, const void* X, const void* W1t, const void* W2t,
                                    const int32_t* ids, const float* weights, const void* dY, void* work, void* dX,
                                    void* dW1t, void* dW2t, float* dweights, cusync_stream_t stream) {
  Layer L;
  cusync_status_t st = read_desc(d, &L, true);
  if (st != CUSYNC_OK) return st;
  if (!aligned(dW1t) || !aligned(dW2t)) return CUSYNC_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (L.T == 0) {  // no token: every weight gradient is zero
    cudaError_t e = cudaMemsetAsync(dW1t, 0, (size_t)L.E * L.G * L.N1 * L.D * 2, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(dW2t, 0, (size_t)L.E * L.N1 * L.D * 2, s);
    if (e == cudaSuccess) e = clear_error(work, s);
    return status_of(e);
  }
  if (!aligned(X) || !aligned(W1t) || !aligned(W2t) || !aligned(ids) || !aligned(weights) || !aligned(dY) ||
      !aligned(work) || !aligned(dX) || !aligned(dweights))
    return CUSYNC_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = prepare_device(&sms)) != CUSYNC_OK) return st;
  if (d->num_sms) sms = std::min(sms, d->num_sms);
  char* w = static_cast<char*>(work);
  const int64_t H = L.G * L.N1;
  // the weights' gradients take pairs where either has more rows than one CTA's tile
  const bool pair = use_pairs(L, sms), pair_g = std::max(H, L.D) > 128 && sms >= 2;
  void *gx = w + L.gx, *gy = w + L.gy, *gh = w + L.gh, *gz = w + L.gz;
  void* rows = w + L.grows;
  float* part = reinterpret_cast<float*>(w + L.gpart);

  GemmArgs p = gemm_args(L, work, weights);  // hidden layer and its gradient
  p.M = (int32_t)L.N1;
  p.K = (int32_t)L.D;
  p.part = part;
  p.parts = L.parts;
  GemmArgs x = gemm_args(L, work, weights);  // dX per slot
  x.M = (int32_t)L.D;
  x.K = (int32_t)H;
  x.out = rows;
  x.scale = reinterpret_cast<uint8_t*>(w + L.gscales);
  GemmArgs g = gemm_args(L, work, weights);  // the weights' gradients
  g.M = (int32_t)H;
  g.N = (int32_t)L.D;
  g.M2 = (int32_t)L.D;
  g.N2 = (int32_t)L.N1;
  const bool wide = L.D % 64 == 0 && L.N1 % 64 == 0;
  p.wide = x.wide = g.wide = wide;
  // a weight gradient's stage holds two blocks of 64 rows on pairs, one on single CTAs
  const int kr = wide && pair_g ? 128 : 64;
  const int last = pair ? kMidRows / 2 : 128;  // BWD1's highest token box
  // BWD1's stage holds one block, DX's two
  if (!map_gate_up(&p.mA, W1t, L.E, L.G, L.N1, L.D, wide) || !map_weights(&p.mA2, W2t, L.E, L.D, L.N1, 64, wide, 2) ||
      !map_hidden(&p.mO, gz, L.S, L.G, L.N1) || !map_hidden(&p.mO2, gh, L.S, 1, L.N1) ||
      !map_tokens(p.mB, gx, L.S, L.D, wide, 1, last) || !map_tokens(p.mB2, gy, L.S, L.D, wide, 1, last) ||
      !map_weights(&x.mA, W1t, L.E, H, L.D, wide ? 128 : 64, wide, 2) || !map_tokens(x.mB, gz, L.S, H, wide, 2) ||
      !map_output(&x.mO, rows, L.S, L.D, 32) || !map_gradient(&g.mO, dW1t, L.E, H, L.D) ||
      !map_gradient(&g.mO2, dW2t, L.E, L.D, L.N1) ||
      !map_rows(&g.mA, gz, L.S, H, kr, wide, 2) || !map_rows(&g.mB[0], gx, L.S, L.D, kr, wide, 2) ||
      !map_rows(&g.mA2, gy, L.S, L.D, kr, wide, 2) || !map_rows(&g.mB2[0], gh, L.S, L.N1, kr, wide, 2))
    return CUSYNC_ERR_CUDA;
  cudaError_t e = launch_plan(L, ids, work, s);
  if (e == cudaSuccess) e = launch_dispatch(L, work, X, gx, dY, gy, s);
  if (e == cudaSuccess)
    e = L.G == 2 ? launch_gemm<BWD1, 1>(pair, p, L, sms, s) : launch_gemm<BWD1, 0>(pair, p, L, sms, s);
  if (e == cudaSuccess) e = launch_gemm<DX, 0>(pair, x, L, sms, s);
  if (e == cudaSuccess) e = launch_combine(L, work, rows, w + L.gscales, nullptr, dX, part, dweights, s);
  if (e == cudaSuccess) e = launch_gemm<DW, 0>(pair_g, g, L, sms, s);
  return status_of(e);
}

cusync_status_t cusync_moe_check(const void* buffer, cusync_stream_t stream, uint32_t* code) {
  if (!aligned(buffer)) return CUSYNC_ERR_INVALID_ARG;
  // a wait inside a capture would end the capture
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing((cudaStream_t)stream, &capture);
  if (e == cudaErrorStreamCaptureImplicit || (e == cudaSuccess && capture != cudaStreamCaptureStatusNone))
    return CUSYNC_ERR_UNSUPPORTED;
  uint32_t err = 0;
  if (e == cudaSuccess) e = cudaMemcpyAsync(&err, buffer, 4, cudaMemcpyDeviceToHost, (cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return CUSYNC_ERR_CUDA;
  if (code) *code = err;
  return err ? CUSYNC_ERR_DEVICE : CUSYNC_OK;
}

}  // extern "C"
