// router_grad_api.cu -- the C ABI of what trains a router (moe_router_grad.h): argument
// checks and launches.
#include "api_checks.cuh"
#include "router_grad.cuh"

namespace moe {
namespace {

bool tokens_ok(const moe_tokens *t, uint32_t k) {
  if (!t || t->S < 1 || t->S > 65535 || (!t->seq && t->S != 1) || !is_aligned(t->seq, 4))
    return false;
  return (uint64_t)t->T * k <= (1u << 30);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_balance_workspace_size(const moe_router *r, uint32_t T, uint32_t S) {
  return router_ok(r) ? balance_ws(*r, T, S) : 0;
}

moe_status moe_balance(const moe_router *r, const void *logits, moe_dtype dt, size_t ld,
                       const int32_t *idx, const moe_tokens *t, float coef, int32_t *count,
                       int32_t *tokens, float *prob, float *loss, void *ws, size_t ws_bytes,
                       void *stream) {
  if (!router_ok(r) || !dtype_ok(dt) || !tokens_ok(t, r->top_k)) return MOE_ERR_INVALID_ARG;
  if (!count || !tokens || !prob || !loss || !is_aligned(count, 4) || !is_aligned(tokens, 4) ||
      !is_aligned(prob, 4) || !is_aligned(loss, 4))
    return MOE_ERR_INVALID_ARG;
  if (t->T > 0 && (!rows_ok(logits, dt, ld, t->T, r->n_expert) || !idx || !is_aligned(idx, 4)))
    return MOE_ERR_INVALID_ARG;
  if (!ws || !is_aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < balance_ws(*r, t->T, t->S)) return MOE_ERR_WORKSPACE;
  return status_of(launch_balance({*r, logits, dt, ld, idx, *t, coef}, count, tokens, prob, loss,
                                  ws, (cudaStream_t)stream));
}

moe_status moe_route_backward(const moe_router *r, const void *logits, moe_dtype dt, size_t ld,
                              const int32_t *idx, const float *dw, const moe_tokens *t,
                              const int32_t *count, const int32_t *tokens, const float *dloss,
                              float coef, void *dlogits, moe_dtype odt, size_t ldd,
                              void *stream) {
  if (!router_ok(r) || !dtype_ok(dt) || !dtype_ok(odt) || !t) return MOE_ERR_INVALID_ARG;
  if (count ? !tokens_ok(t, r->top_k) : (uint64_t)t->T * r->top_k > (1u << 30))
    return MOE_ERR_INVALID_ARG;
  if (t->T == 0) return MOE_OK;
  if (!rows_ok(logits, dt, ld, t->T, r->n_expert) || !rows_ok(dlogits, odt, ldd, t->T, r->n_expert))
    return MOE_ERR_INVALID_ARG;
  if (dw && (!idx || !is_aligned(idx, 4) || !is_aligned(dw, 4))) return MOE_ERR_INVALID_ARG;
  if (count && (!tokens || !is_aligned(count, 4) || !is_aligned(tokens, 4) ||
                !is_aligned(dloss, 4)))
    return MOE_ERR_INVALID_ARG;
  return status_of(launch_route_backward({*r, logits, dt, ld, idx, *t, coef}, dw, count, tokens,
                                         dloss, dlogits, odt, ldd, (cudaStream_t)stream));
}

moe_status moe_combine_backward(const void *dy, moe_dtype ydt, size_t ldy, const void *o,
                                moe_dtype dt, size_t ldo, uint32_t R, const float *w,
                                const int32_t *pos, uint32_t T, uint32_t top_k, uint32_t d,
                                float *dw, void *dout, size_t ldd, void *stream) {
  if (!dtype_ok(dt) || !dtype_ok(ydt)) return MOE_ERR_INVALID_ARG;
  if (top_k < 1 || top_k > 32 || d < 1 || d > (1u << 24) || R > (1u << 30) ||
      (uint64_t)T * top_k > (1u << 30))
    return MOE_ERR_INVALID_ARG;
  if (T == 0 || (!dw && !dout)) return MOE_OK;
  if (!rows_ok(dy, ydt, ldy, T, d) || !pos || !is_aligned(pos, 4)) return MOE_ERR_INVALID_ARG;
  if (dw && (!is_aligned(dw, 4) || (R > 0 && !rows_ok(o, dt, ldo, R, d))))
    return MOE_ERR_INVALID_ARG;
  if (dout && (!w || !is_aligned(w, 4) || (R > 0 && !rows_ok(dout, dt, ldd, R, d))))
    return MOE_ERR_INVALID_ARG;
  return status_of(launch_combine_backward(dy, ydt, ldy, o, dt, ldo, R, w, pos, T, top_k, d, dw,
                                           dout, ldd, (cudaStream_t)stream));
}

}  // extern "C"
