/*
 * moe_fp8.h -- C ABI of the block-scaled fp8 experts and their router
 * (libmoe.so, beside the layer of moe.h).
 *
 * A second weight format for a routed layer, as checkpoints in 8-bit floating
 * point store it: e4m3 codes with one fp32 scale per block of 128 x 128
 * weights, activations quantised to e4m3 with one scale per row and 128
 * columns.  The operators of such a layer, each a call of its own:
 *   moe_group_route   group-limited top-k routing and the row permutation
 *   moe_fp8_quantize  rows to e4m3 codes and block scales
 *   moe_fp8_swiglu    gate and up products of the routed rows, silu(g)*u, codes
 *   moe_fp8_product   out = rows x weights^T, routed or dense
 *   moe_fp8_combine   y[t] = shared[t] + sum_j w[t,j] * o[pos[t,j]]
 *
 * Notation: B = 128, nb(n) = ceil(n / 128).  A matrix X [rows][n] in this
 * format is a code plane of e4m3 bytes [rows][n] (no padding between rows) and
 * a scale plane fp32: X[i][j] = q[i][j] * scale.  The last block of a row may
 * be short.
 *
 * Memory, streams and errors follow moe.h: caller-owned device memory, nothing
 * allocated, asynchronous on `stream`, arguments checked on the host before
 * anything is enqueued.  Each kernel waits for the stream's earlier work before
 * it reads.  Calls that take a workspace need one that was zero-filled when it
 * was allocated; its first MOE_WS_FIXED_BYTES hold the device error word and
 * counters as in moe.h (a workspace of moe_layer serves, if large enough, and
 * calls that overlap need workspaces of their own); moe_check_device_error
 * reads the word.
 */
#ifndef MOE_FP8_H
#define MOE_FP8_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_DT_F32 = 0, MOE_DT_BF16 = 1, MOE_DT_F16 = 2 } moe_dtype;

/* Scoring by softmax over all experts, p_e = e^(l_e - max l) / sum; a value of
 * moe_router.score beside moe_score's (moe_desc does not take it). */
#define MOE_SCORE_SOFTMAX 2

/* A group's score: the largest c of its experts, or the sum of its two largest
 * (its only one where the groups hold one expert). */
typedef enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2_SUM = 1 } moe_group_score;

typedef struct {
  uint32_t n_expert;    /* E, 1..1024 */
  uint32_t top_k;       /* k, 1..32 */
  uint32_t n_group;     /* G, 1..32, divides E; 1 = no groups */
  uint32_t topk_group;  /* groups kept, 1..G; topk_group * E/G >= k */
  uint32_t score;       /* moe_score or MOE_SCORE_SOFTMAX */
  uint32_t group_score; /* moe_group_score */
  uint32_t renorm;      /* 1: weights sum to s; 0: w_j = s * p_j */
  float s;              /* routing scale */
} moe_router;

/* Group-limited routing.  For every token t:
 *   p_e = score of logits[t][e], in fp32 with CUDA's expf (sigmoid
 *         1/(1+e^-l), sqrt(softplus(l)), or softmax);
 *   c_e = p_e + bias[e]; with softmax, no bias and MOE_GROUP_MAX, c_e = l_e
 *         (softmax keeps the order of the logits);
 *   the topk_group groups of E/G consecutive experts with the best group score
 *   are kept (equal scores: the lower group), the k best c among their experts
 *   are picked in descending order (equal c: the lower expert);
 *   w_j = s * p_j / sum_j p_j (renorm) or s * p_j; 0 where the sum is 0.
 * A NaN logit counts as -inf, a NaN c likewise; a -inf logit has p = 0 (also
 * where every logit of the row is), and +inf counts as the largest finite
 * float.  Experts of groups that are not kept are never picked.
 * logits: [T] rows of E values of type dt, row stride ld >= E in elements, aligned
 * to its type.  bias: fp32 [E] or NULL.  Outputs as moe_route's, 4-byte
 * aligned: idx [T][k], w [T][k] fp32, off [E+1], perm [T*k], pos [T*k]: the rows
 * of an expert in (token, slot) order.  T = 0 writes off = 0.
 * ws: moe_group_route_workspace_size bytes (0 for a bad router), 256-byte
 * aligned. */
size_t moe_group_route_workspace_size(const moe_router *r, uint32_t T);
moe_status moe_group_route(const moe_router *r, const void *logits, moe_dtype dt, size_t ld,
                           const float *bias, uint32_t T, int32_t *idx, float *w, int32_t *off,
                           int32_t *perm, int32_t *pos, void *ws, size_t ws_bytes, void *stream);

/* x [T] rows of d values of type dt (row stride ld >= d in elements, aligned to
 * its type) -> q [T][d] e4m3 bytes, scale [T][nb(d)] fp32.  Per row and block
 * of 128 columns: a = max(max|x|, 2^-100), q = rn_e4m3(x * (448 / a)) (saturating,
 * ties to even), scale = a / 448.  A NaN gives a NaN code and leaves the
 * block's scale to its other values; an infinity makes the whole block's values
 * NaN in a product. */
moe_status moe_fp8_quantize(const void *x, moe_dtype dt, size_t ld, uint32_t T, uint32_t d,
                            void *q, float *scale, void *stream);

/* Weights of E experts: q [E][N][K] e4m3 bytes, scale [E][nb(N)][nb(K)] fp32. */
typedef struct {
  const void *q;
  const float *scale;
} moe_fp8_mat;

/* The activation rows of a product and which expert takes them.  Output row r
 * belongs to expert e with off[e] <= r < off[e+1] and reads activation row
 * perm[r] / top_k (perm as moe_group_route's; NULL: row r itself).  off NULL: every
 * row goes to expert 0 (a dense product; n_expert must be 1).  off may start
 * above 0 and end below `rows` (the share of some of the experts: off + e0 and
 * those experts' weights): the other output rows are left as they are.  An off
 * that is not ascending within [0, rows] flags MOE_ERR_DEVICE_CHECK and writes
 * nothing; a perm[r] that names no activation row flags it and leaves row r's
 * output unspecified. */
typedef struct {
  const void *q;       /* e4m3 [n][K] */
  const float *scale;  /* fp32 [n][nb(K)] */
  uint32_t n;          /* activation rows (>= rows where perm is NULL) */
  uint32_t rows;       /* R: output rows */
  const int32_t *off;  /* [E+1] or NULL */
  const int32_t *perm; /* [R] or NULL */
  uint32_t top_k;      /* >= 1; read only with perm */
} moe_fp8_rows;

/* Workspace bytes of a product over `rows` output rows. */
size_t moe_fp8_workspace_size(uint32_t rows);

/* out[r][n] = sum over blocks kb of 128 of scale_x[kb] * scale_w[n/128][kb] *
 * (sum over the block of q_x * q_w), in fp32 -- the inner sum on the tensor cores,
 * the outer one in ascending kb (a tile whose K is split over CTAs: partial sums
 * added in ascending order; runs repeat bit for bit) -- rounded once to odt.
 * out: row stride ld >= N in elements, aligned to its type.  E 1..1024, any
 * N, K >= 1.  With K a multiple of 16 and code planes aligned to 16 bytes the
 * tensor-core kernel runs; otherwise a plain one. */
moe_status moe_fp8_product(const moe_fp8_mat *w, uint32_t n_expert, uint32_t N, uint32_t K,
                           const moe_fp8_rows *x, void *out, moe_dtype odt, size_t ld, void *ws,
                           size_t ws_bytes, void *stream);

/* g and u as moe_fp8_product with the experts' gate and up weights [E][f][d],
 * h = g / (1 + e^-g) * u in fp32, and h quantised as by moe_fp8_quantize:
 * hq [R][f] e4m3 bytes, hs [R][nb(f)] fp32. */
moe_status moe_fp8_swiglu(const moe_fp8_mat *gate, const moe_fp8_mat *up, uint32_t n_expert,
                          uint32_t f, uint32_t d, const moe_fp8_rows *x, void *hq, float *hs,
                          void *ws, size_t ws_bytes, void *stream);

/* y[t] = shared[t] + sum_j w[t][j] * o[pos[t][j]], summed in fp32 in slot order after
 * the shared row, rounded once to ydt.  o: [R] rows of d values, shared: [T]
 * rows or NULL, both of type dt; row strides ldo, lds, ldy in elements.  A pos
 * outside [0, R) contributes nothing (an expert-parallel rank gives the slots
 * of other ranks pos = -1). */
moe_status moe_fp8_combine(const void *o, moe_dtype dt, size_t ldo, uint32_t R, const float *w,
                           const int32_t *pos, uint32_t T, uint32_t top_k, uint32_t d,
                           const void *shared, size_t lds, void *y, moe_dtype ydt, size_t ldy,
                           void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_FP8_H */
