// fp8_api.cu -- the C ABI of the block-scaled fp8 operators (moe_fp8.h):
// argument checks and launches.
#include "api_checks.cuh"

namespace moe {
namespace {

bool mat_ok(const moe_fp8_mat *m) { return m && m->q && m->scale && is_aligned(m->scale, 4); }

// checks shared by the two products; MOE_OK with x->rows == 0: nothing to do
moe_status check_product(const moe_fp8_mat *w0, const moe_fp8_mat *w1, bool two, uint32_t E,
                         uint32_t N, uint32_t K, const moe_fp8_rows *x, const void *ws,
                         size_t ws_bytes) {
  if (!mat_ok(w0) || (two && !mat_ok(w1)) || !x) return MOE_ERR_INVALID_ARG;
  if (E < 1 || E > 1024 || N < 1 || K < 1 || N > (1u << 24) || K > (1u << 24))
    return MOE_ERR_INVALID_ARG;
  if (!x->off && E != 1) return MOE_ERR_INVALID_ARG;
  if (!is_aligned(x->off, 4) || !is_aligned(x->perm, 4)) return MOE_ERR_INVALID_ARG;
  if (x->rows > (1u << 30) || x->n > (1u << 30)) return MOE_ERR_INVALID_ARG;
  if (x->perm ? x->top_k < 1 : x->n < x->rows) return MOE_ERR_INVALID_ARG;
  // tiles are numbered in 31 bits (the smallest are 32 rows by 128 columns)
  if (((uint64_t)x->rows / 32 + E) * fp8_blocks(N) >= (1ull << 31)) return MOE_ERR_INVALID_ARG;
  if (x->rows == 0) return MOE_OK;
  if (x->n == 0 || !x->q || !x->scale || !is_aligned(x->scale, 4)) return MOE_ERR_INVALID_ARG;
  if (!ws || !is_aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < fp8_gemm_ws(x->rows)) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_group_route_workspace_size(const moe_router *r, uint32_t T) {
  if (!router_ok(r)) return 0;
  (void)T;
  return group_route_ws(*r);
}

moe_status moe_group_route(const moe_router *r, const void *logits, moe_dtype dt, size_t ld,
                           const float *bias, uint32_t T, int32_t *idx, float *w, int32_t *off,
                           int32_t *perm, int32_t *pos, void *ws, size_t ws_bytes, void *stream) {
  if (!router_ok(r) || !dtype_ok(dt)) return MOE_ERR_INVALID_ARG;
  if (!off || !is_aligned(off, 4) || !ws || !is_aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  if (T > 0) {
    if (!rows_ok(logits, dt, ld, T, r->n_expert) || !is_aligned(bias, 4))
      return MOE_ERR_INVALID_ARG;
    if (!idx || !w || !perm || !pos) return MOE_ERR_INVALID_ARG;
    if (!is_aligned(idx, 4) || !is_aligned(w, 4) || !is_aligned(perm, 4) || !is_aligned(pos, 4))
      return MOE_ERR_INVALID_ARG;
  }
  if ((uint64_t)T * r->top_k > (1u << 30)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < group_route_ws(*r)) return MOE_ERR_WORKSPACE;
  return status_of(launch_group_route(*r, logits, dt, ld, bias, T, idx, w, off, perm, pos, ws,
                                      (cudaStream_t)stream));
}

moe_status moe_fp8_quantize(const void *x, moe_dtype dt, size_t ld, uint32_t T, uint32_t d,
                            void *q, float *scale, void *stream) {
  if (!dtype_ok(dt) || d < 1 || d > (1u << 24) || T > (1u << 30)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!rows_ok(x, dt, ld, T, d) || !q || !scale || !is_aligned(scale, 4))
    return MOE_ERR_INVALID_ARG;
  // one warp per 8 blocks: the grid's CTAs are numbered in 31 bits
  if ((uint64_t)T * (fp8_blocks(d) / 8 + 1) >= (1ull << 32)) return MOE_ERR_INVALID_ARG;
  return status_of(launch_fp8_quantize(x, dt, ld, T, d, q, scale, (cudaStream_t)stream));
}

size_t moe_fp8_workspace_size(uint32_t rows) { return fp8_gemm_ws(rows); }

moe_status moe_fp8_product(const moe_fp8_mat *w, uint32_t n_expert, uint32_t N, uint32_t K,
                           const moe_fp8_rows *x, void *out, moe_dtype odt, size_t ld, void *ws,
                           size_t ws_bytes, void *stream) {
  if (!dtype_ok(odt)) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_product(w, nullptr, false, n_expert, N, K, x, ws, ws_bytes);
  if (st != MOE_OK || x->rows == 0) return st;
  if (!rows_ok(out, odt, ld, x->rows, N)) return MOE_ERR_INVALID_ARG;
  Fp8Call c = {};
  c.swiglu = false;
  c.w[0] = *w;
  c.E = n_expert;
  c.N = N;
  c.K = K;
  c.x = *x;
  c.out = out;
  c.odt = odt;
  c.ld = ld;
  c.ws = (uint8_t *)ws;
  c.stream = (cudaStream_t)stream;
  return status_of(launch_fp8_gemm(c));
}

moe_status moe_fp8_swiglu(const moe_fp8_mat *gate, const moe_fp8_mat *up, uint32_t n_expert,
                          uint32_t f, uint32_t d, const moe_fp8_rows *x, void *hq, float *hs,
                          void *ws, size_t ws_bytes, void *stream) {
  const moe_status st = check_product(gate, up, true, n_expert, f, d, x, ws, ws_bytes);
  if (st != MOE_OK || x->rows == 0) return st;
  if (!hq || !hs || !is_aligned(hs, 4)) return MOE_ERR_INVALID_ARG;
  Fp8Call c = {};
  c.swiglu = true;
  c.w[0] = *gate;
  c.w[1] = *up;
  c.E = n_expert;
  c.N = f;
  c.K = d;
  c.x = *x;
  c.out = hq;
  c.ld = f;
  c.hs = hs;
  c.ws = (uint8_t *)ws;
  c.stream = (cudaStream_t)stream;
  return status_of(launch_fp8_gemm(c));
}

moe_status moe_fp8_combine(const void *o, moe_dtype dt, size_t ldo, uint32_t R, const float *w,
                           const int32_t *pos, uint32_t T, uint32_t top_k, uint32_t d,
                           const void *shared, size_t lds, void *y, moe_dtype ydt, size_t ldy,
                           void *stream) {
  if (!dtype_ok(dt) || !dtype_ok(ydt)) return MOE_ERR_INVALID_ARG;
  if (top_k < 1 || top_k > 32 || d < 1 || d > (1u << 24) || T > (1u << 30) || R > (1u << 30))
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (R > 0 && !rows_ok(o, dt, ldo, R, d)) return MOE_ERR_INVALID_ARG;
  if (shared && !rows_ok(shared, dt, lds, T, d)) return MOE_ERR_INVALID_ARG;
  if (!rows_ok(y, ydt, ldy, T, d) || !w || !pos || !is_aligned(w, 4) || !is_aligned(pos, 4))
    return MOE_ERR_INVALID_ARG;
  if ((uint64_t)T * ((d + 255) / 256) >= (1ull << 31)) return MOE_ERR_INVALID_ARG;
  return status_of(launch_fp8_combine(o, dt, ldo, R, w, pos, T, top_k, d, shared, lds, y, ydt, ldy,
                                      (cudaStream_t)stream));
}

}  // extern "C"
