// The router's kernels for bf16 logits.
#include "moe_route.cuh"

namespace cusync {
namespace moe {

cudaError_t route_bf16(const RouteArgs& a, bool softmax, bool grad, int sms, cudaStream_t s) {
  return route_logits<__nv_bfloat16>(a, softmax, grad, sms, s);
}

}  // namespace moe
}  // namespace cusync
