// Kernel launches shared by the expert layer's translation units.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace cusync {
namespace moe {

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;        // route: out; gradient: dweights (in)
  void* dlogits;
  int64_t T;
  int32_t E, k, groups, group_size, group_limit, group_top;
  int32_t renorm;
  float scale;
};

// The router's kernels by the logits' type, a translation unit each.
cudaError_t route_f32(const RouteArgs& a, bool softmax, bool grad, int sms, cudaStream_t s);
cudaError_t route_bf16(const RouteArgs& a, bool softmax, bool grad, int sms, cudaStream_t s);

// Every launch is a programmatic dependent of the kernel before it in the stream: it may be
// set up while that one ends, and each kernel waits for that end before it touches memory.
template <typename... P, typename... Q>
cudaError_t launch_cluster(int cluster, void (*f)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, Q... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, f, args...);
}
template <typename... P, typename... Q>
cudaError_t launch(void (*f)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, Q... args) {
  return launch_cluster(1, f, grid, threads, smem, s, args...);
}

}  // namespace moe
}  // namespace cusync
