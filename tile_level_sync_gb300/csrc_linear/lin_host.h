// What the host sides of the norm and of the linear layer share.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/cusync_linear.h"
#include "../csrc_moe/moe_launch.h"
#include "lin_plan.h"

namespace cusync {
namespace lin {

constexpr int64_t kHeader = 256;  // bytes of a work buffer before its arrays; a linear call's error word first

using moe::launch;
using moe::launch_cluster;

inline int64_t round_up(int64_t a, int64_t b) { return div_up(a, b) * b; }
inline bool aligned(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned_or_null(const void* p) { return !p || aligned(p); }
inline cusync_status_t status_of(cudaError_t e) { return e == cudaSuccess ? CUSYNC_OK : CUSYNC_ERR_CUDA; }

}  // namespace lin
}  // namespace cusync
