// router_math.cuh -- a router's logits as the router and its gradients count them.
#pragma once

#include <float.h>

#include "fp8_common.cuh"

namespace moe {

__device__ __forceinline__ float no_nan(float v) { return v == v ? v : -INFINITY; }

// NaN as -inf, +inf as the largest finite value
__device__ __forceinline__ float logit_value(float v) { return fminf(no_nan(v), FLT_MAX); }

}  // namespace moe
