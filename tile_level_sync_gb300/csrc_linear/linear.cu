// Host side of the linear layer in include/cusync_linear.h: argument checks, buffer layouts, TMA
// descriptors and kernel launches.
#include <cudaTypedefs.h>

#include <atomic>
#include <cstring>
#include <mutex>

#include "lin_dz.cuh"
#include "lin_gemm.cuh"
#include "lin_host.h"
#include "lin_plan.h"
#include "lin_split.cuh"

using namespace cusync;
using namespace cusync::lin;

namespace {

constexpr int64_t kDzBlocks = 1024;  // blocks of the pass over dY, about
constexpr int64_t kDzRows = 32;      // rows of such a block at least
constexpr int64_t kResident = 48 << 20;  // bytes of an operand that the L2 (129 MB on two dies) keeps beside what passes by

// What a descriptor means.
struct Layer {
  int64_t M, K, N, G, blocks;
  int64_t dz_pitch, x_pitch;               // of the gradient's own operands: rows begin with a line of 128 bytes
  bool e4m3;
  int64_t dz_rows, dz_parts;               // rows of a block of the pass over dY; blocks along M
  int64_t dz, x, part, work_bytes, grad_bytes;  // gradient work, bytes
};

cusync_status_t read_desc(const cusync_linear_desc_t* d, Layer* L) {
  if (!d || d->M < 0 || d->K < 1 || d->N < 1 || d->num_sms < 0 || d->act < CUSYNC_LINEAR_NONE ||
      d->act > CUSYNC_LINEAR_SWIGLU || (d->dtype != CUSYNC_LINEAR_BF16 && d->dtype != CUSYNC_LINEAR_E4M3))
    return CUSYNC_ERR_INVALID_ARG;
  L->e4m3 = d->dtype == CUSYNC_LINEAR_E4M3;
  // the kernels count rows, columns, tiles and blocks in 32 bits; a tensor map's strides are below 2^40 bytes
  if (d->N % 8 || d->K % (L->e4m3 ? 16 : 8) || d->K > (1 << 24) || d->N > (1 << 24) || d->M > (1 << 30) ||
      d->K * d->N >= (int64_t)1 << 38 ||
      div_up(d->M, 16) * div_up(std::max(d->N, d->K), 64) > INT32_MAX / 8 ||
      div_up(2 * d->N, 64) * div_up(d->K, 64) > INT32_MAX / 8 || div_up(d->M * d->K, 1 << 15) > INT32_MAX / 2)
    return CUSYNC_ERR_UNSUPPORTED;
  L->M = d->M;
  L->K = d->K;
  L->N = d->N;
  L->G = d->act == CUSYNC_LINEAR_SWIGLU ? 2 : 1;
  L->blocks = div_up(d->N, kBlock);
  L->dz_pitch = round_up(L->G * L->N, 64);
  L->x_pitch = round_up(L->K, 64);
  const int64_t columns = div_up(L->N, kDzCols);
  L->dz_rows = std::max(kDzRows, round_up(div_up(L->M, std::max<int64_t>(1, kDzBlocks / columns)), 8));
  L->dz_parts = std::max<int64_t>(1, div_up(L->M, L->dz_rows));
  int64_t b = kHeader;
  auto bytes = [&b](int64_t n) {
    const int64_t at = b;
    b += round_up(n, 256);
    return at;
  };
  L->work_bytes = b;
  L->dz = bytes(d->act == CUSYNC_LINEAR_NONE && !L->e4m3 ? 0 : L->M * L->dz_pitch * 2);
  L->x = bytes(L->e4m3 ? L->M * L->x_pitch * 2 : 0);
  L->part = bytes(L->dz_parts * L->G * L->N * 4);
  L->grad_bytes = b;
  return CUSYNC_OK;
}

// ----------------------------------------------------------------------------- devices

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::mutex g_mu;
constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];  // SMs of a prepared device, 0 = not prepared

cudaError_t prepare_kernel(const void* f, int smem) {
  cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;  // loads the kernel now, not at its first launch
  return cudaFuncGetAttributes(&fa, f);
}
template <int MODE, bool E4M3, bool GATED, int BN>
cudaError_t prepare_gemm() {
  return prepare_kernel(reinterpret_cast<const void*>(&gemm_kernel<MODE, E4M3, GATED, BN>), GemmCfg<MODE, GATED, BN>::kSmem);
}
template <int MODE, bool E4M3, bool GATED>
cudaError_t prepare_split() {
  return prepare_kernel(reinterpret_cast<const void*>(&split_kernel<MODE, E4M3, GATED>), kSmemPerSm - 1024);
}
template <bool E4M3, bool GATED>
cudaError_t prepare_forward() {
  cudaError_t e = prepare_gemm<FWD, E4M3, GATED, 256>();
  if (e == cudaSuccess) e = prepare_gemm<FWD, E4M3, GATED, 128>();
  return e == cudaSuccess ? prepare_split<FWD, E4M3, GATED>() : e;
}

// The current device: the attributes set of the kernels that need some, the descriptor encoder
// found.  The first call on a device does the work.
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
  if (e == cudaSuccess) e = prepare_forward<false, false>();
  if (e == cudaSuccess) e = prepare_forward<false, true>();
  if (e == cudaSuccess) e = prepare_forward<true, false>();
  if (e == cudaSuccess) e = prepare_forward<true, true>();
  if (e == cudaSuccess) e = prepare_gemm<GRAD, false, false, 256>();
  if (e == cudaSuccess) e = prepare_gemm<GRAD, false, false, 128>();
  if (e == cudaSuccess) e = prepare_split<DX, false, false>();
  if (e == cudaSuccess) e = prepare_split<DW, false, false>();
  if (e != cudaSuccess) return CUSYNC_ERR_CUDA;
  g_sms[dev].store(n, std::memory_order_release);
  *sms = n;
  return CUSYNC_OK;
}

// A map of `bytes`-wide elements: sizes and strides (in elements, from the second dimension on) and
// the box, innermost first; elements outside read as zero.  Rows that begin inside a line of 128 bytes make a box's row
// two of them, of which the L2 should not fetch four (4096 x K x 4096 in e4m3, us with lines fetched by twos / alone: K
// 8048 129 / 118, 8032 102 / 95; 8064, a multiple of 128, 84 / 84).
template <int N>
bool map_nd(CUtensorMap* m, const void* p, int bytes, CUtensorMapSwizzle swizzle, const int64_t (&size)[N],
            const int64_t (&stride)[N - 1], const int (&box_size)[N]) {
  cuuint64_t dims[N], strides[N - 1];
  cuuint32_t box[N], one[N];
  for (int i = 0; i < N; ++i) {
    dims[i] = (cuuint64_t)size[i];
    box[i] = (cuuint32_t)box_size[i];
    one[i] = 1;
    if (i) strides[i - 1] = (cuuint64_t)stride[i - 1] * bytes;
  }
  return g_encode(m, bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, N,
                  const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  stride[0] * bytes % 128 ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An operand [rows, cols], rows `pitch` elements apart, whose columns are the reduction's: boxes of 128 bytes x
// box_rows; wide (columns a multiple of 128 bytes): as [blocks][rows][128 bytes], boxes of two.
bool map_rows(CUtensorMap* m, const void* p, int bytes, int64_t rows, int64_t cols, int64_t pitch, int box_rows,
              int32_t* wide) {
  const int n = 128 / bytes;
  *wide = cols % n == 0;
  return *wide ? map_nd<3>(m, p, bytes, CU_TENSOR_MAP_SWIZZLE_128B, {n, rows, cols / n}, {pitch, n}, {n, box_rows, 2})
               : map_nd<2>(m, p, bytes, CU_TENSOR_MAP_SWIZZLE_128B, {cols, rows}, {pitch}, {n, box_rows});
}
// Gate and up rows of a gated layer's weights [2][rows, cols], 64 of each in a box.
bool map_gated(CUtensorMap* m, const void* p, int bytes, int64_t rows, int64_t cols, int32_t* wide) {
  const int n = 128 / bytes;
  *wide = cols % n == 0;
  return *wide ? map_nd<4>(m, p, bytes, CU_TENSOR_MAP_SWIZZLE_128B, {n, rows, 2, cols / n}, {cols, rows * cols, n},
                           {n, 64, 2, 2})
               : map_nd<3>(m, p, bytes, CU_TENSOR_MAP_SWIZZLE_128B, {cols, rows, 2}, {cols, rows * cols}, {n, 64, 2});
}
// A bf16 operand [rows, cols] whose rows are the reduction's: boxes of 64 columns x 128 rows; wide (columns
// a multiple of 64): as [chunks][rows][64], boxes of `chunks`.
bool map_along(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t pitch, int chunks,
               int32_t* wide) {
  *wide = cols % 64 == 0;
  return *wide ? map_nd<3>(m, p, 2, CU_TENSOR_MAP_SWIZZLE_128B, {64, rows, cols / 64}, {pitch, 64}, {64, 128, chunks})
               : map_nd<2>(m, p, 2, CU_TENSOR_MAP_SWIZZLE_128B, {cols, rows}, {pitch}, {64, 128});
}
// An output [rows, cols]: boxes of 32 x 32 as a warp's lanes write them.
bool map_output(CUtensorMap* m, void* p, int64_t rows, int64_t cols) {
  return map_nd<2>(m, p, 2, CU_TENSOR_MAP_SWIZZLE_64B, {cols, rows}, {cols}, {32, 32});
}

// ----------------------------------------------------------------------------- products

// One product: `rows` x `cols` outputs (SwiGLU: columns of Y), reduction `depth`.  P and Q are the
// operands of the output's rows and columns: [rows, depth] and [cols, depth] (SwiGLU: [2 * cols, depth]),
// or, where they lie along the output, [depth, rows] and [depth, cols]; their rows are p_pitch and q_pitch elements
// apart.
struct Product {
  const void *P, *Q;
  int64_t rows, cols, depth, p_pitch, q_pitch;
  Epilogue e;
};

template <int MODE, bool E4M3, bool GATED>
cudaError_t launch_split(const Plan& plan, const Product& p, int32_t* err, bool clear, cudaStream_t s) {
  constexpr int bytes = E4M3 ? 1 : 2;
  SplitArgs a;
  std::memset(&a, 0, sizeof(a));
  a.e = p.e;
  a.err = err;
  a.clear = clear;
  a.M = (int32_t)p.rows;
  a.N = (int32_t)p.cols;
  a.K = (int32_t)p.depth;
  a.cols = plan.cols;
  a.row_tiles = (int32_t)div_up(p.rows, plan.cols);
  a.b_rows = MODE == DW ? plan.cols : (int32_t)std::min<int64_t>(plan.cols, round_up(p.rows, 8));
  a.splits = plan.splits;
  a.stages = plan.stages;
  a.apart = plan.apart;
  const bool ok = (MODE != FWD  ? map_along(&a.mA, p.Q, p.depth, p.cols, p.q_pitch, 2, &a.wideA)
                   : GATED      ? map_gated(&a.mA, p.Q, bytes, p.cols, p.depth, &a.wideA)
                                : map_rows(&a.mA, p.Q, bytes, p.cols, p.depth, p.q_pitch, 128, &a.wideA)) &&
                  (MODE == DW ? map_along(&a.mB, p.P, p.depth, p.rows, p.p_pitch, plan.cols / 64, &a.wideB)
                              : map_rows(&a.mB, p.P, bytes, p.rows, p.depth, p.p_pitch, a.b_rows, &a.wideB));
  if (!ok) return cudaErrorInvalidValue;
  const int64_t tiles = div_up(p.cols, GATED ? 64 : 128) * a.row_tiles;
  return launch_cluster(plan.splits, split_kernel<MODE, E4M3, GATED>, dim3((unsigned)(tiles * plan.splits)), kSplitThreads,
                        split_smem(plan.cols, plan.stages, plan.apart), s, a);
}

// A product on pairs; along: P's rows are the reduction's (dWt).  Q's are, too, in both gradients.
template <int MODE, bool E4M3, bool GATED, int BN>
bool fill_shape(GemmShape* g, const Product& p, bool along) {
  constexpr int bytes = E4M3 ? 1 : 2;
  g->M = (int32_t)p.rows;
  g->N = (int32_t)p.cols;
  g->K = (int32_t)p.depth;
  g->m_tiles = (int32_t)div_up(p.rows, 256);
  g->n_tiles = (int32_t)div_up(p.cols, GATED ? BN / 2 : BN);
  // Row tiles whose A stays in the L2 while the columns' B passes by: as few groups as such a share allows, and B
  // marked to leave first where one group is all and both do not fit.  Under the power cap bytes from HBM cost
  // MMAs (us of passes for seconds; groups of 2, 4, 8, 16 row tiles, 29 to 34 MB of A in 16: SwiGLU 4096 x 8192 x 3584 in
  // e4m3 158, 157, 156, 153, linear 4096 x 3584 x 8192 169, 163, 160, 157, with B leaving first 149 and 154.5; both gradients
  // of the first, 59 MB in 16 and in 28: 650, 629, 615, 618; by shares of 20, 36, 48, 64 MB 611, 610, 607, 623).
  const int64_t a_bytes = p.rows * p.depth * bytes, b_bytes = p.cols * (GATED ? 2 : 1) * p.depth * bytes;
  const int64_t groups = std::min<int64_t>(std::max<int64_t>(1, div_up(a_bytes, kResident)), g->m_tiles);
  g->group = (int32_t)div_up(g->m_tiles, groups);
  g->b_first = MODE == FWD && groups == 1 && a_bytes + b_bytes > 3 * kResident / 2;
  g->along = along;
  g->a_rows = along ? 128 : (int32_t)std::min<int64_t>(128, round_up(p.rows, 8));
  return (along ? map_along(&g->mA, p.P, p.depth, p.rows, p.p_pitch, 2, &g->wideA)
                : map_rows(&g->mA, p.P, bytes, p.rows, p.depth, p.p_pitch, g->a_rows, &g->wideA)) &&
         (MODE == GRAD ? map_along(&g->mB, p.Q, p.depth, p.cols, p.q_pitch, BN / 128, &g->wideB)
               : map_rows(&g->mB, p.Q, bytes, GATED ? 2 * p.cols : p.cols, p.depth, p.q_pitch, BN / 2, &g->wideB)) &&
         map_output(&g->mO, p.e.out, p.rows, p.cols);
}
template <int MODE, bool E4M3, bool GATED, int BN>
cudaError_t launch_gemm(const GemmArgs& a, int sms, cudaStream_t s) {
  const int64_t tiles = (int64_t)a.p[0].m_tiles * a.p[0].n_tiles + (int64_t)a.p[1].m_tiles * a.p[1].n_tiles;
  const unsigned grid = 2 * (unsigned)std::min<int64_t>(tiles, sms / 2);
  return launch_cluster(2, gemm_kernel<MODE, E4M3, GATED, BN>, dim3(grid), GemmCfg<MODE, GATED, BN>::kThreads, GemmCfg<MODE, GATED, BN>::kSmem, s, a);
}

template <bool E4M3, bool GATED>
cudaError_t forward(const Product& p, int32_t* err, int sms, cudaStream_t s) {
  constexpr int elems = E4M3 ? 128 : 64;
  const Plan pair = pair_plan(p.rows, p.cols, p.depth, sms, elems, GATED);
  const Plan split = split_plan<FWD, GATED>(p.rows, p.cols, p.depth, sms, elems);
  if (split.us <= pair.us) return launch_split<FWD, E4M3, GATED>(split, p, err, true, s);
  GemmArgs a;
  std::memset(&a, 0, sizeof(a));
  a.e = p.e;
  a.err = err;
  a.clear = true;
  if (p.e.R && !map_output(&a.mR, const_cast<uint16_t*>(p.e.R), p.rows, p.cols)) return cudaErrorInvalidValue;
  if (pair.bn == 256)
    return fill_shape<FWD, E4M3, GATED, 256>(&a.p[0], p, false) ? launch_gemm<FWD, E4M3, GATED, 256>(a, sms, s)
                                                                  : cudaErrorInvalidValue;
  return fill_shape<FWD, E4M3, GATED, 128>(&a.p[0], p, false) ? launch_gemm<FWD, E4M3, GATED, 128>(a, sms, s)
                                                                : cudaErrorInvalidValue;
}

// dX and dWt (either may be NULL), and on pairs dbias's sums.
struct Sums {
  const float* part;
  uint16_t* out;
  int64_t rows, cols;
};
template <int BN>
cudaError_t pair_gradients(const Product* dx, const Product* dw, const Sums& sums, int32_t* err, bool clear, int sms,
                           cudaStream_t s) {
  GemmArgs a;
  std::memset(&a, 0, sizeof(a));
  a.err = err;
  a.clear = clear;
  a.part = sums.part;
  a.sums = sums.out;
  a.part_rows = (int32_t)sums.rows;
  a.part_cols = (int32_t)sums.cols;
  if (dx) a.e.Xs = dx->e.Xs;
  const bool dw_first = dw && (!dx || dw->depth > dx->depth);
  GemmShape *gx = &a.p[dw_first ? 1 : 0], *gw = &a.p[dw_first || !dx ? 0 : 1];
  if ((dx && !fill_shape<GRAD, false, false, BN>(gx, *dx, false)) || (dw && !fill_shape<GRAD, false, false, BN>(gw, *dw, true)))
    return cudaErrorInvalidValue;
  return launch_gemm<GRAD, false, false, BN>(a, sms, s);
}
cudaError_t sum_columns(const Sums& sums, cudaStream_t s) {
  return launch(column_sum_kernel, dim3((unsigned)div_up(sums.cols, 32)), 256, 0, s, sums.part, (int32_t)sums.rows,
                (int32_t)sums.cols, sums.out);
}
// Both on pairs in one launch, or one or both on clusters: what is estimated fastest.
cudaError_t gradients(const Product* dx, const Product* dw, const Sums& sums, int32_t* err, bool clear, int sms,
                      cudaStream_t s) {
  Plan px = {0}, pw = {0}, sx = {0}, sw = {0};
  if (dx) {
    px = pair_plan(dx->rows, dx->cols, dx->depth, sms, 64, false);
    sx = split_plan<DX, false>(dx->rows, dx->cols, dx->depth, sms, 64);
  }
  if (dw) {
    pw = pair_plan(dw->rows, dw->cols, dw->depth, sms, 64, false);
    sw = split_plan<DW, false>(dw->rows, dw->cols, dw->depth, sms, 64);
  }
  int bn = dx && px.us < sx.us ? px.bn : 0;  // of the launch on pairs
  bool split_x = dx && !bn, split_w = dw && sw.us <= pw.us;
  if (dw && !split_w) bn = bn ? std::min(bn, pw.bn) : pw.bn;
  if (dx && dw && sms >= 2) {
    double apart = std::min(px.us, sx.us) + std::min(pw.us, sw.us);
    for (int n = 128; n <= 256; n += 128) {
      const int64_t tx = div_up(dx->rows, 256) * div_up(dx->cols, n), tw = div_up(dw->rows, 256) * div_up(dw->cols, n);
      const double ux = pair_tile(n, div_up(dx->depth, 64)), uw = pair_tile(n, div_up(dw->depth, 64));
      const double us = ux > uw ? pair_time(tx, ux, tw, uw, sms / 2) : pair_time(tw, uw, tx, ux, sms / 2);
      if (us < apart) {
        apart = us;
        bn = n;
        split_x = split_w = false;
      }
    }
  }
  cudaError_t e = cudaSuccess;
  if (sums.part && !bn) e = sum_columns(sums, s);
  if (e == cudaSuccess && split_x) {
    e = launch_split<DX, false, false>(sx, *dx, err, clear, s);
    clear = false;
  }
  if (e == cudaSuccess && split_w) {
    e = launch_split<DW, false, false>(sw, *dw, err, clear, s);
    clear = false;
  }
  if (e == cudaSuccess && bn) {
    const Product *x = split_x ? nullptr : dx, *w = split_w ? nullptr : dw;
    e = bn == 256 ? pair_gradients<256>(x, w, sums, err, clear, sms, s) : pair_gradients<128>(x, w, sums, err, clear, sms, s);
  }
  return e;
}

cusync_status_t capture_or_ok(cudaStream_t s) {
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  const cudaError_t e = cudaStreamIsCapturing(s, &capture);
  if (e == cudaErrorStreamCaptureImplicit || (e == cudaSuccess && capture != cudaStreamCaptureStatusNone))
    return CUSYNC_ERR_UNSUPPORTED;
  return status_of(e);
}

}  // namespace

extern "C" {

cusync_status_t cusync_linear_info(const cusync_linear_desc_t* d, cusync_linear_info_t* out) {
  Layer L;
  if (!out) return CUSYNC_ERR_INVALID_ARG;
  const cusync_status_t st = read_desc(d, &L);
  if (st != CUSYNC_OK) return st;
  out->work_bytes = L.work_bytes;
  out->grad_work_bytes = L.grad_bytes;
  out->parts = L.G;
  out->blocks = L.blocks;
  return CUSYNC_OK;
}

cusync_status_t cusync_linear(const cusync_linear_desc_t* d, const void* X, const float* Xs, const void* Wt,
                              const float* Ws, const void* bias, const void* R, void* work, void* Y, void* Zq,
                              uint8_t* Ze, cusync_stream_t stream) {
  Layer L;
  cusync_status_t st = read_desc(d, &L);
  if (st != CUSYNC_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (!aligned(work) || (L.M && !Zq != !Ze) || (!L.e4m3 && (Xs || Ws))) return CUSYNC_ERR_INVALID_ARG;
  if (L.M == 0) return status_of(cudaMemsetAsync(work, 0, 4, s));
  if (!aligned(X) || !aligned(Wt) || !aligned(Y) || !aligned_or_null(bias) || !aligned_or_null(R) ||
      !aligned_or_null(Zq) || !aligned_or_null(Ze) || (L.e4m3 && (!aligned(Xs) || !aligned(Ws))))
    return CUSYNC_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = prepare_device(&sms)) != CUSYNC_OK) return st;
  if (d->num_sms) sms = std::min(sms, d->num_sms);
  Product p = {};
  p.P = X;
  p.Q = Wt;
  p.rows = L.M;
  p.cols = L.N;
  p.depth = p.p_pitch = p.q_pitch = L.K;
  p.e.Xs = Xs;
  p.e.Ws = Ws;
  p.e.bias = static_cast<const uint16_t*>(bias);
  p.e.R = static_cast<const uint16_t*>(R);
  p.e.Zq = static_cast<uint8_t*>(Zq);
  p.e.Ze = Ze;
  p.e.out = static_cast<uint16_t*>(Y);
  p.e.act = d->act;
  int32_t* err = static_cast<int32_t*>(work);
  return status_of(L.e4m3 ? (L.G == 2 ? forward<true, true>(p, err, sms, s) : forward<true, false>(p, err, sms, s))
                          : (L.G == 2 ? forward<false, true>(p, err, sms, s) : forward<false, false>(p, err, sms, s)));
}

cusync_status_t cusync_linear_grad(const cusync_linear_desc_t* d, const void* X, const float* Xs, const void* Wt,
                                   const void* Zq, const uint8_t* Ze, const void* dY, void* work, void* dX,
                                   void* dWt, void* dbias, cusync_stream_t stream) {
  Layer L;
  cusync_status_t st = read_desc(d, &L);
  if (st != CUSYNC_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  const bool act = d->act != CUSYNC_LINEAR_NONE;
  if (!aligned(work) || (L.M && !dX && !dWt && !dbias) || !aligned_or_null(dX) || !aligned_or_null(dWt) ||
      !aligned_or_null(dbias) || (!L.e4m3 && Xs))
    return CUSYNC_ERR_INVALID_ARG;
  const int64_t H = L.G * L.N;
  if (L.M == 0) {  // no token: the parameters' gradients are zero
    cudaError_t e = cudaMemsetAsync(work, 0, 4, s);
    if (e == cudaSuccess && dWt) e = cudaMemsetAsync(dWt, 0, (size_t)H * L.K * 2, s);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, (size_t)H * 2, s);
    return status_of(e);
  }
  if (!aligned(dY) || (act && (!aligned(Zq) || !aligned(Ze))) || (dX && !aligned(Wt)) ||
      (dWt && (!aligned(X) || (L.e4m3 && !aligned(Xs)))))
    return CUSYNC_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = prepare_device(&sms)) != CUSYNC_OK) return st;
  if (d->num_sms) sms = std::min(sms, d->num_sms);
  char* w = static_cast<char*>(work);
  int32_t* err = static_cast<int32_t*>(work);
  bool clear = true;
  cudaError_t e = cudaSuccess;
  // 8-bit X: dWt's operand is dZ times the fractions of its scales, and dX's the same but where dY itself will do
  const bool scaled = L.e4m3 && dWt;
  const void* dZ = act ? w + L.dz : dY;
  if (act || dbias || scaled) {
    DzArgs a = {};
    a.dY = static_cast<const uint16_t*>(dY);
    a.Zq = static_cast<const uint8_t*>(Zq);
    a.Ze = Ze;
    a.dZ = scaled || (act && (dX || dWt)) ? reinterpret_cast<uint16_t*>(w + L.dz) : nullptr;
    if (scaled) {
      a.Xs = Xs;
      a.q = static_cast<const uint4*>(X);
      a.x = reinterpret_cast<uint4*>(w + L.x);
      a.pieces = L.M * (L.K / 16);
      a.row_pieces = (int32_t)(L.K / 16);
      a.x_pitch = L.x_pitch;
    }
    a.part = dbias ? reinterpret_cast<float*>(w + L.part) : nullptr;
    a.err = err;
    a.M = L.M;
    a.N = (int32_t)L.N;
    a.dz_pitch = L.dz_pitch;
    a.rows = (int32_t)L.dz_rows;
    a.col_blocks = (int32_t)div_up(L.N, kDzCols);
    a.parts = (int32_t)L.dz_parts;
    clear = false;
    const dim3 grid((unsigned)(a.col_blocks * L.dz_parts + div_up(a.pieces, 256 * kUnpackPieces)));
    e = d->act == CUSYNC_LINEAR_NONE   ? launch(dz_kernel<ACT_NONE>, grid, 256, 0, s, a)
        : d->act == CUSYNC_LINEAR_RELU ? launch(dz_kernel<ACT_RELU>, grid, 256, 0, s, a)
        : d->act == CUSYNC_LINEAR_GELU ? launch(dz_kernel<ACT_GELU>, grid, 256, 0, s, a)
                                       : launch(dz_kernel<ACT_SWIGLU>, grid, 256, 0, s, a);
  }
  Product dx = {}, dw = {};
  dx.P = dZ;
  dx.e.Xs = scaled && act ? Xs : nullptr;
  dw.P = scaled ? w + L.dz : dZ;
  dw.p_pitch = scaled || act ? L.dz_pitch : L.N;
  dw.q_pitch = L.e4m3 ? L.x_pitch : L.K;
  dx.p_pitch = act ? L.dz_pitch : L.N;
  dx.Q = Wt;
  dx.q_pitch = L.K;
  dx.rows = L.M;
  dx.cols = L.K;
  dx.depth = H;
  dx.e.out = static_cast<uint16_t*>(dX);
  dw.Q = L.e4m3 ? w + L.x : X;
  dw.rows = H;
  dw.cols = L.K;
  dw.depth = L.M;
  dw.e.out = static_cast<uint16_t*>(dWt);
  const Sums sums = {dbias ? reinterpret_cast<const float*>(w + L.part) : nullptr, static_cast<uint16_t*>(dbias), L.dz_parts, H};
  if (e == cudaSuccess) e = gradients(dX ? &dx : nullptr, dWt ? &dw : nullptr, sums, err, clear, sms, s);
  return status_of(e);
}

cusync_status_t cusync_linear_check(const void* work, cusync_stream_t stream, uint32_t* code) {
  if (!aligned(work)) return CUSYNC_ERR_INVALID_ARG;
  // a wait inside a capture would end the capture
  const cusync_status_t st = capture_or_ok((cudaStream_t)stream);
  if (st != CUSYNC_OK) return st;
  uint32_t err = 0;
  cudaError_t e = cudaMemcpyAsync(&err, work, 4, cudaMemcpyDeviceToHost, (cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return CUSYNC_ERR_CUDA;
  if (code) *code = err;
  return err ? CUSYNC_ERR_DEVICE : CUSYNC_OK;
}

}  // extern "C"
