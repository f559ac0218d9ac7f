// Host side of the norm in include/cusync_linear.h: argument checks and kernel launches.
#include <atomic>
#include <cmath>

#include "lin_host.h"
#include "lin_norm.cuh"

using namespace cusync;
using namespace cusync::lin;

namespace {

// Blocks of the gradient's kernels, which are the rows of its partial sums.
constexpr int kGradBlocks = 152 * 4;

cusync_status_t read_desc(const cusync_norm_desc_t* d) {
  if (!d || d->M < 0 || d->D < 1 || d->num_sms < 0 || !std::isfinite(d->eps) || d->eps < 0.0f ||
      (d->kind != CUSYNC_NORM_RMS && d->kind != CUSYNC_NORM_NONE))
    return CUSYNC_ERR_INVALID_ARG;
  if (d->D % 8 || d->D > CUSYNC_NORM_MAX_D || d->M > INT32_MAX) return CUSYNC_ERR_UNSUPPORTED;
  return CUSYNC_OK;
}

// Pieces of 8 columns a thread, and threads of a block.
struct Shape {
  int v, threads;
  bool warps;  // of which each warp takes a row
};
// Rows of a block: up to 256 threads with one piece, then more pieces, at most `most` while 1024 threads will do.
// Short rows are warps' from `rows` of them on: fewer are done sooner by more threads each.
Shape shape(int64_t M, int64_t D, int most, int64_t rows) {
  const int64_t vecs = D / 8;
  int v = 1;
  if (vecs <= kWarpVecs && M >= rows) {
    while (32 * v < vecs) v *= 2;
    return {v, kRowWarps * 32, true};
  }
  while (v < 4 && vecs > (v < most ? 256 : 1024) * v) v *= 2;
  return {v, (int)round_up(div_up(vecs, v), 32), false};
}

// Rows of up to 1024 columns from which warps take them (us, blocks / warps: norm 650 rows of 256 1.8 / 1.7, of 1000 1.9 / 2.4;
// 1000 rows of 256 1.9 / 1.7, of 512 2.0 / 1.9, of 1000 2.7 / 2.4 and with residual and 8 bits 2.6 / 2.7; 1777 rows of 1000
// 3.2 / 2.9; gradient of rows of 1000, 32 rows 3.5 / 4.7, 333 5.5 / 4.9, 1000 9.0 / 5.5).
constexpr int64_t kNormWarpRows = 1000, kGradWarpRows = 256;

// The gradient's blocks on an SM, and rows of a ring (a block's, or each of its warps').
struct Ring {
  int per_sm, stages;
  size_t bytes;  // of a block
};
constexpr int kRingBytes = 208 * 1024;  // of an SM
Ring ring(int64_t D, const Shape& s, bool ds) {
  const int row = (int)D * 2 * (ds && (s.warps || s.v < 4) ? 3 : 2) * (s.warps ? kRowWarps : 1);
  const int per_sm = s.warps ? 2 : s.v == 1 ? 4 : s.v == 2 && s.threads <= 256 ? 3 : 1;  // as their registers allow
  const int stages = std::min(kNormStages, std::max(1, kRingBytes / per_sm / row));
  return {per_sm, stages, std::max((size_t)stages * row, s.warps ? (size_t)D * 4 * kRowWarps : 0)};
}

constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];  // SMs of a prepared device, 0 = not prepared

const void* grad_kernel(const Shape& s) {
  if (s.warps)
    return reinterpret_cast<const void*>(s.v == 1   ? &norm_grad_warp_kernel<1>
                                         : s.v == 2 ? &norm_grad_warp_kernel<2>
                                                    : &norm_grad_warp_kernel<4>);
  return reinterpret_cast<const void*>(s.v == 1                       ? &norm_grad_block_kernel<1, 256, 4>
                                       : s.v == 2 && s.threads <= 256 ? &norm_grad_block_kernel<2, 256, 3>
                                       : s.v == 2 && s.threads <= 512 ? &norm_grad_block_kernel<2, 512, 1>
                                       : s.v == 2 && s.threads <= 768 ? &norm_grad_block_kernel<2, 768, 1>
                                       : s.v == 2                     ? &norm_grad_block_kernel<2, 1024, 1>
                                       : s.threads <= 768             ? &norm_grad_block_kernel<4, 768, 1>
                                                                      : &norm_grad_block_kernel<4, 1024, 1>);
}

// The current device, the gradient's kernels set up.  The first call on a device does the work.
cusync_status_t prepare_device(int* sms) {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) return CUSYNC_ERR_CUDA;
  if ((*sms = g_sms[dev].load(std::memory_order_acquire))) return CUSYNC_OK;
  cudaError_t e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  const Shape all[] = {{1, 0, true}, {2, 0, true}, {4, 0, true}, {1, 256, false},
                       {2, 256, false}, {2, 512, false}, {2, 768, false}, {2, 1024, false}, {4, 768, false},
                       {4, 1024, false}};
  for (const Shape& s : all)
    if (e == cudaSuccess) e = cudaFuncSetAttribute(grad_kernel(s), cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (e != cudaSuccess) return CUSYNC_ERR_CUDA;
  g_sms[dev].store(*sms = n, std::memory_order_release);
  return CUSYNC_OK;
}

}  // namespace

extern "C" {

cusync_status_t cusync_norm_info(const cusync_norm_desc_t* d, cusync_norm_info_t* out) {
  if (!out) return CUSYNC_ERR_INVALID_ARG;
  const cusync_status_t st = read_desc(d);
  if (st != CUSYNC_OK) return st;
  out->grad_work_bytes = kHeader + round_up(std::min<int64_t>(std::max<int64_t>(d->M, 1), kGradBlocks) * d->D * 4, 256);
  return CUSYNC_OK;
}

cusync_status_t cusync_norm(const cusync_norm_desc_t* d, const void* X, const void* R, const void* w, void* S,
                            void* Y, void* Q, float* Qs, cusync_stream_t stream) {
  const cusync_status_t st = read_desc(d);
  if (st != CUSYNC_OK) return st;
  const bool rms = d->kind == CUSYNC_NORM_RMS;
  if (d->M == 0) return CUSYNC_OK;
  if ((!S && !Y && !Q) || !Q != !Qs) return CUSYNC_ERR_INVALID_ARG;
  if (!aligned(X) || (rms && !aligned(w)) || !aligned_or_null(R) || !aligned_or_null(S) || !aligned_or_null(Y) ||
      !aligned_or_null(Q) || !aligned_or_null(Qs))
    return CUSYNC_ERR_INVALID_ARG;
  NormArgs a = {};
  a.X = static_cast<const uint4*>(X);
  a.R = static_cast<const uint4*>(R);
  a.w = static_cast<const uint4*>(w);
  a.S = static_cast<uint4*>(S);
  a.Y = static_cast<uint4*>(Y);
  a.Q = static_cast<uint2*>(Q);
  a.Qs = Qs;
  a.M = d->M;
  a.vecs = (int32_t)(d->D / 8);
  a.rms = rms;
  a.eps = d->eps;
  a.inv_d = 1.0f / (float)d->D;
  const Shape s = shape(d->M, d->D, 4, kNormWarpRows);
  cudaStream_t q = (cudaStream_t)stream;
  if (s.warps) {
    const dim3 grid((unsigned)div_up(d->M, kRowWarps));
    return status_of(s.v == 1   ? launch(norm_warp_kernel<1>, grid, s.threads, 0, q, a)
                     : s.v == 2 ? launch(norm_warp_kernel<2>, grid, s.threads, 0, q, a)
                                : launch(norm_warp_kernel<4>, grid, s.threads, 0, q, a));
  }
  const dim3 grid((unsigned)d->M);
  return status_of(s.v == 1           ? launch(norm_block_kernel<1, 256>, grid, s.threads, 0, q, a)
                   : s.v == 2         ? launch(norm_block_kernel<2, 256>, grid, s.threads, 0, q, a)
                   : s.threads <= 256 ? launch(norm_block_kernel<4, 256>, grid, s.threads, 0, q, a)
                   : s.threads <= 512 ? launch(norm_block_kernel<4, 512>, grid, s.threads, 0, q, a)
                                      : launch(norm_block_kernel<4, 1024>, grid, s.threads, 0, q, a));
}

cusync_status_t cusync_norm_grad(const cusync_norm_desc_t* d, const void* S, const void* w, const void* dY,
                                 const void* dS, void* work, void* dX, void* dw, cusync_stream_t stream) {
  const cusync_status_t st = read_desc(d);
  if (st != CUSYNC_OK) return st;
  if (d->kind != CUSYNC_NORM_RMS) return CUSYNC_ERR_UNSUPPORTED;
  cudaStream_t q = (cudaStream_t)stream;
  if (!aligned_or_null(dw)) return CUSYNC_ERR_INVALID_ARG;
  if (!aligned(work)) return CUSYNC_ERR_INVALID_ARG;
  if (d->M == 0) {
    cudaError_t e = cudaMemsetAsync(work, 0, 4, q);
    if (e == cudaSuccess && dw) e = cudaMemsetAsync(dw, 0, (size_t)d->D * 2, q);
    return status_of(e);
  }
  if (!aligned(S) || !aligned(w) || !aligned(dY) || !aligned_or_null(dS) || !aligned(dX)) return CUSYNC_ERR_INVALID_ARG;
  int sms = 0;
  const cusync_status_t ready = prepare_device(&sms);
  if (ready != CUSYNC_OK) return ready;
  if (d->num_sms) sms = std::min(sms, d->num_sms);
  NormGradArgs a = {};
  a.S = static_cast<const uint4*>(S);
  a.w = static_cast<const uint4*>(w);
  a.dY = static_cast<const uint4*>(dY);
  a.dS = static_cast<const uint4*>(dS);
  a.dX = static_cast<uint4*>(dX);
  a.part = dw ? reinterpret_cast<float*>(static_cast<char*>(work) + kHeader) : nullptr;
  a.err = static_cast<int32_t*>(work);
  a.M = d->M;
  a.vecs = (int32_t)(d->D / 8);
  a.eps = d->eps;
  a.inv_d = 1.0f / (float)d->D;
  const Shape s = shape(d->M, d->D, 2, kGradWarpRows);
  const Ring g = ring(d->D, s, dS != nullptr);
  a.stages = g.stages;
  // Each block writes a row of sums, at half a row's cost and more, and they are read again: four rows of the
  // gradient a block at least, while every SM has one.
  const int64_t units = s.warps ? div_up(d->M, kRowWarps) : d->M;
  const int blocks = (int)std::min<int64_t>(std::min<int64_t>(units, kGradBlocks),
                                            std::min<int64_t>((int64_t)sms * g.per_sm, std::max<int64_t>(sms, div_up(units, 4))));
  const dim3 grid((unsigned)blocks);
  cudaError_t e;
  if (s.warps)
    e = s.v == 1   ? launch(norm_grad_warp_kernel<1>, grid, s.threads, g.bytes, q, a)
        : s.v == 2 ? launch(norm_grad_warp_kernel<2>, grid, s.threads, g.bytes, q, a)
                   : launch(norm_grad_warp_kernel<4>, grid, s.threads, g.bytes, q, a);
  else
    e = s.v == 1                       ? launch(norm_grad_block_kernel<1, 256, 4>, grid, s.threads, g.bytes, q, a)
        : s.v == 2 && s.threads <= 256 ? launch(norm_grad_block_kernel<2, 256, 3>, grid, s.threads, g.bytes, q, a)
        : s.v == 2 && s.threads <= 512 ? launch(norm_grad_block_kernel<2, 512, 1>, grid, s.threads, g.bytes, q, a)
        : s.v == 2 && s.threads <= 768 ? launch(norm_grad_block_kernel<2, 768, 1>, grid, s.threads, g.bytes, q, a)
        : s.v == 2                     ? launch(norm_grad_block_kernel<2, 1024, 1>, grid, s.threads, g.bytes, q, a)
        : s.threads <= 768             ? launch(norm_grad_block_kernel<4, 768, 1>, grid, s.threads, g.bytes, q, a)
                                       : launch(norm_grad_block_kernel<4, 1024, 1>, grid, s.threads, g.bytes, q, a);
  if (e == cudaSuccess && dw)
    e = launch(column_sum_kernel, dim3((unsigned)div_up(d->D, 32)), 256, 0, q, (const float*)a.part, (int32_t)blocks,
               (int32_t)d->D, static_cast<uint16_t*>(dw));
  return status_of(e);
}

}  // extern "C"
