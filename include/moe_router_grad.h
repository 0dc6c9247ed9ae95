/*
 * moe_router_grad.h -- C ABI of what trains a router (libmoe.so): the loss that
 * evens out the experts' load, and the gradients that reach the router's logits
 * through the routing weights and through that loss.
 *   moe_balance           per-expert counts, mean probabilities and the loss
 *   moe_route_backward    the logits' gradient
 *   moe_combine_backward  gradients of the weighted combine
 * The experts' weights take no gradient; the picks (idx) are constants.
 *
 * Notation: E, k, s, scores p_e of a token's logits and weights w_j of its picks as
 * moe_group_route defines them (moe_router; its groups play no part here, and what
 * it does with NaN and infinite logits holds here too; its sigmoid is 0 below -88.72283,
 * and so is p_e; its sqrt(softplus), whose e^l is a subnormal number from -87 and 0 from
 * -103.97 down, is here that of the exact e^l down to -174);
 *   share_e = p_e (softmax) or p_e / sum_e p_e, 0 where the sum is 0.
 *
 * Sequences: seq [S+1] ascending token offsets in [0, T]; sequence i's tokens are
 * seq[i] .. seq[i+1] - 1, tokens before seq[0] and from seq[S] on belong to none.  seq
 * NULL: S = 1, all T tokens.  live [T]: bytes, 0 marks padding; NULL: none.  A token
 * counts if it is live and of a sequence; n_i is how many of sequence i do (it may
 * be 0).  Of a seq that is not ascending within [0, T] it is unspecified which tokens
 * count; nothing outside the arrays is touched.
 *
 * Memory, streams, errors and the workspace follow moe_fp8.h.  Sums are held in
 * fp32 in a fixed order: calls repeat bit for bit.
 */
#ifndef MOE_ROUTER_GRAD_H
#define MOE_ROUTER_GRAD_H

#include "moe_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The tokens of a call and which of them count. */
typedef struct {
  uint32_t T;          /* tokens */
  uint32_t S;          /* sequences, 1 .. 65535 */
  const int32_t *seq;  /* [S+1], or NULL with S = 1 */
  const uint8_t *live; /* [T] or NULL */
} moe_tokens;

/* count[i][e] = picks of expert e by sequence i's counting tokens (a pick outside
 *               [0, E) is none's; the same expert twice in a token counts twice);
 * tokens[i]   = n_i;
 * prob[i][e]  = sum of share_e over them / n_i, 0 where n_i is 0;
 * loss[0]     = coef / S * sum over i of sum over e of f[i][e] * prob[i][e],
 *               f[i][e] = E * count[i][e] / (k * n_i), 0 where n_i is 0.
 * logits: [T] rows of E values of type dt, row stride ld.  idx [T][k] as
 * moe_group_route's.  count [S][E] int32, tokens [S] int32, prob [S][E] fp32, loss
 * fp32 [1].  ws: moe_balance_workspace_size bytes (0 for a bad router). */
size_t moe_balance_workspace_size(const moe_router *r, uint32_t T, uint32_t S);
moe_status moe_balance(const moe_router *r, const void *logits, moe_dtype dt, size_t ld,
                       const int32_t *idx, const moe_tokens *t, float coef, int32_t *count,
                       int32_t *tokens, float *prob, float *loss, void *ws, size_t ws_bytes,
                       void *stream);

/* dlogits[t][e] = d/dlogits[t][e] of (sum over j of dw[t][j] * w[t][j] + dloss * loss):
 *   slope_e (share_e (a_e - sum a share) + [e picked] v_j),  slope = d log p / dl
 *   a_e = dloss * coef / S * E * count[i][e] / (k n_i^2), 0 for tokens that do not count
 *   v_j = s q_j (dw_j - sum dw q), q_j = p_j / sum of the picks' p (renorm), or
 *   s p_j dw_j (softmax: and the sum of all picks' v times p_e is taken off every expert).
 * dw [T][k] fp32, or NULL: no such part.  count [S][E] and tokens [S] as moe_balance
 * wrote them, or count NULL: no such part (seq, live, dloss and coef are not read).  dloss: fp32 [1] on the
 * device, NULL counts as 1.  live and seq say which tokens the loss's part reaches; dw's
 * reaches all.  A pick outside [0, E) takes no part.  dlogits: [T] rows of E values of
 * type odt, row stride ldd; it may be logits itself if the types and strides are alike. */
moe_status moe_route_backward(const moe_router *r, const void *logits, moe_dtype dt, size_t ld,
                              const int32_t *idx, const float *dw, const moe_tokens *t,
                              const int32_t *count, const int32_t *tokens, const float *dloss,
                              float coef, void *dlogits, moe_dtype odt, size_t ldd, void *stream);

/* Gradients of y[t] = shared[t] + sum_j w[t][j] * o[pos[t][j]] (moe_fp8_combine):
 *   dw[t][j] = sum over d of dy[t] * o[pos[t][j]], in fp32; 0 where pos is outside [0, R);
 *   dout[pos[t][j]] = w[t][j] * dy[t], rounded once to dt (shared's gradient is dy itself).
 * A row of o is in at most one slot, as moe_group_route's pos has it: what dout has of a
 * row that several slots name is unspecified; rows that none names are left as they are.
 * o: [R] rows of d values of type dt, stride ldo; dy: [T] rows of type ydt, stride ldy.
 * dw [T][k] or NULL (o is then not read); dout: [R] rows of type dt, stride ldd, or NULL (w
 * is then not read).  dout must not overlap o or dy. */
moe_status moe_combine_backward(const void *dy, moe_dtype ydt, size_t ldy, const void *o,
                                moe_dtype dt, size_t ldo, uint32_t R, const float *w,
                                const int32_t *pos, uint32_t T, uint32_t top_k, uint32_t d,
                                float *dw, void *dout, size_t ldd, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_ROUTER_GRAD_H */
