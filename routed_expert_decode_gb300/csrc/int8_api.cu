// int8_api.cu -- the C ABI of the int8 operators (moe_int8.h): argument checks and
// launches.
#include "api_checks.cuh"
#include "int8.cuh"

namespace moe {
namespace {

constexpr uint32_t kMaxK = 131071;  // 2^14 K stays below 2^31

bool mat_ok(const moe_int8_mat *m) { return m && m->q && m->scale && is_aligned(m->scale, 4); }

// the two products; w1: SwiGLU's second matrix
moe_status product(const moe_int8_mat *w0, const moe_int8_mat *w1, bool two, uint32_t E,
                   uint32_t N, uint32_t K, const moe_int8_rows *x, void *out, moe_dtype odt,
                   size_t ld, void *ws, size_t ws_bytes, void *stream) {
  if (!dtype_ok(odt) || !mat_ok(w0) || (two && !mat_ok(w1)) || !x) return MOE_ERR_INVALID_ARG;
  if (E < 1 || E > 1024 || N < 1 || K < 1 || N > (1u << 24) || K > kMaxK)
    return MOE_ERR_INVALID_ARG;
  if (!x->off && E != 1) return MOE_ERR_INVALID_ARG;
  if (!is_aligned(x->off, 4) || !is_aligned(x->perm, 4)) return MOE_ERR_INVALID_ARG;
  if (x->rows > (1u << 30) || x->n > (1u << 30)) return MOE_ERR_INVALID_ARG;
  if (x->perm ? x->top_k < 1 : x->n < x->rows) return MOE_ERR_INVALID_ARG;
  // tiles are numbered in 31 bits (the smallest are 32 rows by 64 columns)
  if (((uint64_t)x->rows / 32 + E) * (N / 64 + 1) >= (1ull << 31)) return MOE_ERR_INVALID_ARG;
  if (x->rows == 0) return MOE_OK;
  if (x->n == 0 || !x->q || !x->scale || !is_aligned(x->scale, 4)) return MOE_ERR_INVALID_ARG;
  if (!rows_ok(out, odt, ld, x->rows, N)) return MOE_ERR_INVALID_ARG;
  if (!ws || !is_aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < int8_gemm_ws()) return MOE_ERR_WORKSPACE;
  Int8Call c = {};
  c.swiglu = two;
  c.w[0] = *w0;
  if (two) c.w[1] = *w1;
  c.E = E;
  c.N = N;
  c.K = K;
  c.x = *x;
  c.out = out;
  c.odt = odt;
  c.ld = ld;
  c.ws = (uint8_t *)ws;
  c.stream = (cudaStream_t)stream;
  return status_of(launch_int8_gemm(c));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_int8_quantize(const void *x, moe_dtype dt, size_t ld, uint32_t T, uint32_t d,
                             void *q, float *scale, void *stream) {
  if (!dtype_ok(dt) || d < 1 || d > (1u << 24) || T > (1u << 30)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!rows_ok(x, dt, ld, T, d) || !q || !scale || !is_aligned(scale, 4))
    return MOE_ERR_INVALID_ARG;
  return status_of(launch_int8_quantize(x, dt, ld, T, d, q, scale, (cudaStream_t)stream));
}

// the same for any number of rows: what the shares of split tiles take
size_t moe_int8_workspace_size(uint32_t) { return int8_gemm_ws(); }

moe_status moe_int8_product(const moe_int8_mat *w, uint32_t n_expert, uint32_t N, uint32_t K,
                            const moe_int8_rows *x, void *out, moe_dtype odt, size_t ld, void *ws,
                            size_t ws_bytes, void *stream) {
  return product(w, nullptr, false, n_expert, N, K, x, out, odt, ld, ws, ws_bytes, stream);
}

moe_status moe_int8_swiglu(const moe_int8_mat *gate, const moe_int8_mat *up, uint32_t n_expert,
                           uint32_t f, uint32_t d, const moe_int8_rows *x, void *h, moe_dtype odt,
                           size_t ld, void *ws, size_t ws_bytes, void *stream) {
  return product(gate, up, true, n_expert, f, d, x, h, odt, ld, ws, ws_bytes, stream);
}

}  // extern "C"
