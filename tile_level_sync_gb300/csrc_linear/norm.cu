// Host side of the norm in include/cusync_linear.h: argument checks and kernel launches.
#include <atomic>
#include <cmath>

#include "lin_host.h"
#include "lin_norm.cuh"

using namespace cusync;
using namespace cusync::lin;

namespace {

// Blocks of the gradient's kernel, which are the rows of its partial sums.
constexpr int kGradBlocks = 152 * 8;

cusync_status_t read_desc(const cusync_norm_desc_t* d) {
  if (!d || d->M < 0 || d->D < 1 || d->num_sms < 0 || !std::isfinite(d->eps) || d->eps < 0.0f ||
      (d->kind != CUSYNC_NORM_RMS && d->kind != CUSYNC_NORM_NONE))
    return CUSYNC_ERR_INVALID_ARG;
  if (d->D % 8 || d->D > CUSYNC_NORM_MAX_D || d->M > INT32_MAX) return CUSYNC_ERR_UNSUPPORTED;
  return CUSYNC_OK;
}

// Pieces of 8 columns a thread, and threads of a row's block.
struct Shape {
  int v, threads;
};
// Up to `full` threads with one piece, then more pieces, at most `most` while 1024 threads will do.
Shape shape(int64_t D, int full, int most) {
  const int64_t vecs = D / 8;
  int v = 1;
  while (v < 4 && vecs > (v < most ? full : 1024) * v) v *= 2;
  return {v, (int)round_up(div_up(vecs, v), 32)};
}

// Blocks of the gradient's kernel on an SM, and rows of a block's ring.
struct Ring {
  int per_sm, stages;
};
constexpr int kRingBytes = 208 * 1024;  // of an SM
Ring ring(const cusync_norm_desc_t* d, const Shape& s, int tensors) {
  const int row = (int)d->D * 2 * tensors;
  int per_sm = std::min(8, std::max(1, 1024 / s.threads));
  while (per_sm > 1 && 4 * row > kRingBytes / per_sm) --per_sm;
  return {per_sm, std::min(kNormStages, std::max(1, kRingBytes / per_sm / row))};
}

constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];  // SMs of a prepared device, 0 = not prepared

// The current device, the gradient's kernels set up.  The first call on a device does the work.
cusync_status_t prepare_device(int* sms) {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) return CUSYNC_ERR_CUDA;
  if ((*sms = g_sms[dev].load(std::memory_order_acquire))) return CUSYNC_OK;
  cudaError_t e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  const void* kernels[] = {reinterpret_cast<const void*>(&norm_grad_kernel<1, 256>),
                           reinterpret_cast<const void*>(&norm_grad_kernel<2, 512>),
                           reinterpret_cast<const void*>(&norm_grad_kernel<2, 1024>),
                           reinterpret_cast<const void*>(&norm_grad_kernel<4, 1024>)};
  for (const void* f : kernels)
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
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
  const Shape s = shape(d->D, 256, 4);
  const dim3 grid((unsigned)d->M);
  cudaStream_t q = (cudaStream_t)stream;
  return status_of(s.v == 1         ? launch(norm_kernel<1, 256>, grid, s.threads, 0, q, a)
                   : s.v == 2       ? launch(norm_kernel<2, 256>, grid, s.threads, 0, q, a)
                   : s.threads <= 256 ? launch(norm_kernel<4, 256>, grid, s.threads, 0, q, a)
                   : s.threads <= 512 ? launch(norm_kernel<4, 512>, grid, s.threads, 0, q, a)
                                      : launch(norm_kernel<4, 1024>, grid, s.threads, 0, q, a));
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
  const Shape s = shape(d->D, 256, 2);
  const int tensors = dS ? 3 : 2;
  const Ring g = ring(d, s, tensors);
  a.stages = g.stages;
  const int blocks = (int)std::min<int64_t>(d->M, std::min<int64_t>(kGradBlocks, (int64_t)sms * g.per_sm));
  const dim3 grid((unsigned)blocks);
  const size_t smem = (size_t)g.stages * tensors * d->D * 2;
  cudaError_t e = s.v == 1                       ? launch(norm_grad_kernel<1, 256>, grid, s.threads, smem, q, a)
                  : s.v == 2 && s.threads <= 512 ? launch(norm_grad_kernel<2, 512>, grid, s.threads, smem, q, a)
                  : s.v == 2                     ? launch(norm_grad_kernel<2, 1024>, grid, s.threads, smem, q, a)
                                                 : launch(norm_grad_kernel<4, 1024>, grid, s.threads, smem, q, a);
  if (e == cudaSuccess && dw)
    e = launch(column_sum_kernel, dim3((unsigned)div_up(d->D, 32)), 256, 0, q, (const float*)a.part, (int32_t)blocks,
               (int32_t)d->D, static_cast<uint16_t*>(dw));
  return status_of(e);
}

}  // extern "C"
