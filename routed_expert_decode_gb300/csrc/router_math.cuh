// router_math.cuh -- scores of a router's logits, as the router and its gradients use
// them.
#pragma once

#include <float.h>

#include "fp8_common.cuh"

namespace moe {

// order-preserving map of a float (never NaN) to an unsigned above 0; -0 as +0
__device__ __forceinline__ uint32_t order_key(float c) {
  const uint32_t b = __float_as_uint(c + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ float no_nan(float v) { return v == v ? v : -INFINITY; }

__device__ __forceinline__ float logit_value(float v) { return fminf(no_nan(v), FLT_MAX); }

// sigmoid and sqrt(softplus) with CUDA's expf and log1pf; -inf gives 0
__device__ __forceinline__ float sigmoid_of(float l) { return __frcp_rn(1.0f + expf(-l)); }
__device__ __forceinline__ float softplus_root_of(float l) {
  return __fsqrt_rn(fmaxf(l, 0.0f) + log1pf(expf(-fabsf(l))));
}
// e^(l - max) of a row: 0 at -inf, a row of nothing else included
__device__ __forceinline__ float softmax_term(float l, float m) {
  return l == -INFINITY ? 0.0f : expf(l - m);
}

}  // namespace moe
