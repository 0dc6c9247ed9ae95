// router_grad.cuh -- launchers of what trains a router (moe_router_grad.h)
#pragma once

#include "moe_router_grad.h"
#include "router_math.cuh"

namespace moe {

// word of the workspace's counter area: CTAs of a loss that are done, zero between calls
constexpr uint32_t kBalanceSync = kFp8TileSync + kFp8MaxCtas * 4;
static_assert(kBalanceSync < MOE_SYNC_BYTES / 4 - 2, "counters overlap the layer's");

struct RouterGradArgs {
  moe_router r;
  const void *logits;
  int dt;
  size_t ld;
  const int32_t *idx;
  moe_tokens t;
  float coef;
};

size_t balance_ws(const moe_router &r, uint32_t T, uint32_t S);
cudaError_t launch_balance(const RouterGradArgs &a, int32_t *count, int32_t *tokens, float *prob,
                           float *loss, void *ws, cudaStream_t stream);
cudaError_t launch_route_backward(const RouterGradArgs &a, const float *dw, const int32_t *count,
                                  const int32_t *tokens, const float *dloss, void *dlogits,
                                  int odt, size_t ldd, cudaStream_t stream);
cudaError_t launch_combine_backward(const void *dy, int ydt, size_t ldy, const void *o, int dt,
                                    size_t ldo, uint32_t R, const float *w, const int32_t *pos,
                                    uint32_t T, uint32_t k, uint32_t d, float *dw, void *dout,
                                    size_t ldd, cudaStream_t stream);

}  // namespace moe
