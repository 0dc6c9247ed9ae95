/*
 * moe_int8.h -- C ABI of the int8 experts (libmoe.so, beside the layer of moe.h
 * and the block-scaled fp8 operators of moe_fp8.h).
 *
 * A third weight format for a routed layer, as checkpoints in 8-bit integers
 * with a scale per token and per channel store it: int8 codes with one fp32
 * scale per weight row (output channel), activations quantised to int8 with one
 * scale per row (token).  The operators, each a call of its own:
 *   moe_int8_quantize  rows to int8 codes and row scales
 *   moe_int8_swiglu    gate and up products of the routed rows, silu(g)*u
 *   moe_int8_product   out = rows x weights^T, routed or dense
 * moe_group_route and moe_fp8_combine stand before and behind them.
 *
 * A matrix X [rows][n] in this format is a code plane of int8 [rows][n] (no
 * padding between rows) and fp32 scale [rows]: X[i][j] = q[i][j] * scale[i].
 * Codes are two's complement, -128 .. 127.
 *
 * Memory, streams, errors and the workspace follow moe_fp8.h: caller-owned device
 * memory, nothing allocated, asynchronous on `stream`, arguments checked on the
 * host before anything is enqueued, a workspace that was zero-filled when it was
 * allocated and whose error word moe_check_device_error reads.
 */
#ifndef MOE_INT8_H
#define MOE_INT8_H

#include "moe_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* x [T] rows of d values of type dt (row stride ld >= d in elements, aligned to
 * its type) -> q [T][d] int8, scale [T] fp32.  Per row: a = max(max|x|, 2^-100),
 * q = round(x * (127 / a)) (ties to even), scale = a / 127, each operation in
 * fp32.  A row that holds a NaN or an infinity gets the scale NaN and codes 0, so
 * that every product of the row is NaN.  d up to 2^24. */
moe_status moe_int8_quantize(const void *x, moe_dtype dt, size_t ld, uint32_t T, uint32_t d,
                             void *q, float *scale, void *stream);

/* Weights of E experts: q [E][N][K] int8, scale [E][N] fp32. */
typedef struct {
  const void *q;
  const float *scale;
} moe_int8_mat;

/* The activation rows of a product and which expert takes them: off, perm and
 * top_k, and what a bad off or perm does, as in moe_fp8_rows. */
typedef struct {
  const void *q;       /* int8 [n][K] */
  const float *scale;  /* fp32 [n] */
  uint32_t n;          /* activation rows (>= rows where perm is NULL) */
  uint32_t rows;       /* R: output rows */
  const int32_t *off;  /* [E+1] or NULL */
  const int32_t *perm; /* [R] or NULL */
  uint32_t top_k;      /* >= 1; read only with perm */
} moe_int8_rows;

/* Workspace bytes of a product over `rows` output rows. */
size_t moe_int8_workspace_size(uint32_t rows);

/* out[r][n] = (sum over k of q_x[r][k] * q_w[e][n][k]) * (scale_x[r] * scale_w[e][n]),
 * rounded once to odt.  Runs repeat bit for bit.  out: row stride ld >= N in
 * elements, aligned to its type.  E 1..1024, N up to 2^24, K up to 131071 (a sum
 * of K products fits 32 bits).  With K a multiple of 16 and code planes aligned to
 * 16 bytes the tensor-core kernel runs, or for few rows in all a stream of the
 * weights; otherwise a plain one.
 * The sum is exact wherever no partial sum of its products passes 2^24 in
 * magnitude, and always in the stream and the plain kernel.  On the tensor cores it
 * is held in fp32, whose additions, of 16 products each, cut off what is below an
 * ulp: beyond 2^24 the sum is off by less than 2^-23 K/16 of its products'
 * magnitudes, towards 0 (products of one sign: 3.5e-5 low for K 8208, 9e-4 for
 * 131056).  There the value of a row can differ with the number of rows of a call. */
moe_status moe_int8_product(const moe_int8_mat *w, uint32_t n_expert, uint32_t N, uint32_t K,
                            const moe_int8_rows *x, void *out, moe_dtype odt, size_t ld, void *ws,
                            size_t ws_bytes, void *stream);

/* g and u as moe_int8_product with the experts' gate and up weights [E][f][d], in
 * fp32; h[r][n] = g / (1 + e^-g) * u, rounded once to odt: row stride ld >= f. */
moe_status moe_int8_swiglu(const moe_int8_mat *gate, const moe_int8_mat *up, uint32_t n_expert,
                           uint32_t f, uint32_t d, const moe_int8_rows *x, void *h, moe_dtype odt,
                           size_t ld, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_INT8_H */
