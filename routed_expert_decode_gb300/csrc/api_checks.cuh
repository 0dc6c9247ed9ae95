// api_checks.cuh -- checks of arguments that the operators' C entries share.
#pragma once

#include "fp8_common.cuh"

namespace moe {

inline bool is_aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline bool dtype_ok(int dt) { return dt == MOE_DT_F32 || dt == MOE_DT_BF16 || dt == MOE_DT_F16; }

// rows of n elements at a stride of ld: strides that cannot overflow an offset
inline bool rows_ok(const void *p, int dt, size_t ld, uint32_t rows, uint32_t n) {
  return p && is_aligned(p, dtype_size(dt)) && ld >= n && ld <= ((size_t)1 << 40) &&
         rows <= (1u << 30);
}

inline bool router_ok(const moe_router *r) {
  if (!r) return false;
  if (r->n_expert < 1 || r->n_expert > 1024 || r->top_k < 1 || r->top_k > 32) return false;
  if (r->n_group < 1 || r->n_group > 32 || r->n_expert % r->n_group) return false;
  if (r->topk_group < 1 || r->topk_group > r->n_group) return false;
  if (r->topk_group * (r->n_expert / r->n_group) < r->top_k) return false;
  if (r->score != MOE_SCORE_SIGMOID && r->score != MOE_SCORE_SQRT_SOFTPLUS &&
      r->score != MOE_SCORE_SOFTMAX)
    return false;
  if (r->group_score != MOE_GROUP_MAX && r->group_score != MOE_GROUP_TOP2_SUM) return false;
  if (r->renorm > 1 || !(r->s == r->s)) return false;
  return true;
}

inline moe_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  set_last_error(cudaGetErrorName(e));
  return MOE_ERR_CUDA;
}

}  // namespace moe
