// The router's kernels for fp32 logits.
#include "moe_route.cuh"

namespace cusync {
namespace moe {

cudaError_t route_f32(const RouteArgs& a, bool softmax, bool grad, int sms, cudaStream_t s) {
  return route_logits<float>(a, softmax, grad, sms, s);
}

}  // namespace moe
}  // namespace cusync
