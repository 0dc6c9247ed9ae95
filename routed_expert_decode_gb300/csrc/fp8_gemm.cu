// fp8_gemm.cu -- routed and dense products over e4m3 operands with a scale per
// 128 x 128 weights and per row and 128 activations, on CUDA cores: the kernel
// for operands that tensor copies cannot take (a reduction length that is not a
// multiple of 16, code planes that are not 16-byte aligned).
// Bound by issue: 16384 rows of gate/up of 6144 x 2048 take 33 ms here, 0.34 to 0.39 there.
#include "fp8_tc.cuh"

namespace moe {
namespace {

constexpr int kCoreM = 32, kCoreN = 128;  // rows and columns of a tile
constexpr int kCoreThreads = 256;
constexpr int kCoreSlab = 32;  // K staged at a time

// A tile is 32 rows by one block of 128 columns, so that SwiGLU's outputs of a
// row form whole quantisation blocks in one CTA.  Thread (ty, tx) holds rows
// ty + 8i and columns tx + 32j; 32 K at a time are staged as floats (a row pitch
// of 33 keeps the columns in distinct banks), the sum over a block of 128 is
// kept apart and then scaled, as the definition says.
template <bool SWIGLU>
__global__ void __launch_bounds__(kCoreThreads) k_fp8_core(const Fp8Args a) {
  pdl_trigger();
  pdl_wait();
  constexpr int NM = SWIGLU ? 2 : 1;
  extern __shared__ __align__(16) uint8_t csm[];
  float *sx = (float *)csm;                                // [kCoreM][33]
  float *sw = sx + kCoreM * (kCoreSlab + 1);               // [NM][kCoreN][33]
  int *tiles_sm = (int *)(sw + NM * kCoreN * (kCoreSlab + 1));
  const RowTiles rt = fp8_row_tiles<kCoreM>(a, tiles_sm);
  const int tid = threadIdx.x, tx = tid & 31, ty = tid >> 5;
  const int n_all = rt.total * (int)a.n_tiles;
  for (int v = blockIdx.x; v < n_all; v += gridDim.x) {
    const Fp8Tile t = fp8_tile<kCoreM>(a, rt, v);
    const uint32_t n0 = (uint32_t)t.nt * kCoreN;
    int xrow[4];  // activation rows of this thread's rows, -1: none
#pragma unroll
    for (int i = 0; i < 4; ++i)
      xrow[i] = ty + 8 * i < t.rows ? fp8_x_row(a, t.row0 + ty + 8 * i) : -1;
    float acc[NM][4][4];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][i][j] = 0.0f;
    for (uint32_t kb = 0; kb < a.nbk; ++kb) {
      float part[NM][4][4];
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[m][i][j] = 0.0f;
      for (uint32_t ks = 0; ks < kFp8Block; ks += kCoreSlab) {
        const uint32_t k0 = kb * kFp8Block + ks;
        if (k0 >= a.K) break;
        __syncthreads();
        // row ty + 8i, one of its 32 codes a lane
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool ok = xrow[i] >= 0 && k0 + tx < a.K;
          sx[(ty + 8 * i) * (kCoreSlab + 1) + tx] =
              ok ? e4m3_to_float(a.xq[(size_t)xrow[i] * a.K + k0 + tx]) : 0.0f;
        }
#pragma unroll
        for (int m = 0; m < NM; ++m)
          for (int n = ty; n < kCoreN; n += 8) {
            const bool ok = n0 + n < a.N && k0 + tx < a.K;
            sw[(m * kCoreN + n) * (kCoreSlab + 1) + tx] =
                ok ? e4m3_to_float(a.wq[m][((size_t)t.e * a.N + n0 + n) * a.K + k0 + tx]) : 0.0f;
          }
        __syncthreads();
        for (int q = 0; q < kCoreSlab; ++q) {
          float xv[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) xv[i] = sx[(ty + 8 * i) * (kCoreSlab + 1) + q];
#pragma unroll
          for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float wv = sw[(m * kCoreN + tx + 32 * j) * (kCoreSlab + 1) + q];
#pragma unroll
              for (int i = 0; i < 4; ++i) part[m][i][j] = __fmaf_rn(xv[i], wv, part[m][i][j]);
            }
        }
      }
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const float ws = a.wsc[m][((size_t)t.e * a.nbn + t.nt) * a.nbk + kb];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float s = xrow[i] >= 0 ? ws * a.xs[(size_t)xrow[i] * a.nbk + kb] : 0.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[m][i][j] = __fmaf_rn(part[m][i][j], s, acc[m][i][j]);
        }
      }
    }
    // outputs: a warp (one ty) holds whole rows of the tile
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (ty + 8 * i >= t.rows) continue;  // the same for the warp
      const int r = t.row0 + ty + 8 * i;
      if (!SWIGLU) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n0 + tx + 32 * j < a.N) fp8_store(a, r, n0 + tx + 32 * j, acc[0][i][j]);
      } else {
        float h[4], amax = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[j] = n0 + tx + 32 * j < a.N ? fp8_swiglu_value(acc[0][i][j], acc[NM - 1][i][j]) : 0.0f;
          amax = fmaxf(amax, fabsf(h[j]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float sc, inv;
        fp8_block_scale(amax, sc, inv);
        if (tx == 0) a.hs[(size_t)r * a.nbn + t.nt] = sc;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n0 + tx + 32 * j < a.N)
            ((uint8_t *)a.out)[(size_t)r * a.N + n0 + tx + 32 * j] = e4m3x1(h[j] * inv);
      }
    }
  }
}

template <bool SWIGLU>
cudaError_t run_core(Fp8Args &a, cudaStream_t stream) {
  auto kern = k_fp8_core<SWIGLU>;
  fp8_set_tiles(a, fp8_blocks(a.N), 1);
  const size_t smem = 4 * ((size_t)(kCoreM + (SWIGLU ? 2 : 1) * kCoreN) * (kCoreSlab + 1)) +
                      fp8_tiles_smem(a.E);
  static std::atomic<bool> done[kMaxDevices];
  const cudaError_t e = allow_smem(kern, done);
  if (e != cudaSuccess) return e;
  return launch_k(kern, 4 * fp8_ctas(), kCoreThreads, smem, stream, true, a);
}

}  // namespace

size_t fp8_gemm_ws(uint32_t rows) {
  return MOE_WS_FIXED_BYTES + fp8_tc_ws(rows);
}

cudaError_t launch_fp8_gemm(const Fp8Call &c) {
  Fp8Args a = {};
  a.E = c.E;
  a.N = c.N;
  a.K = c.K;
  a.nbn = fp8_blocks(c.N);
  a.nbk = fp8_blocks(c.K);
  a.n_x = c.x.n;
  a.R = c.x.rows;
  a.top_k = c.x.top_k;
  a.xq = (const uint8_t *)c.x.q;
  a.xs = c.x.scale;
  a.off = c.x.off;
  a.perm = c.x.perm;
  for (int m = 0; m < (c.swiglu ? 2 : 1); ++m) {
    a.wq[m] = (const uint8_t *)c.w[m].q;
    a.wsc[m] = c.w[m].scale;
  }
  a.out = c.out;
  a.ld = c.ld;
  a.hs = c.hs;
  a.odt = c.odt;
  a.err = (uint32_t *)c.ws;
  a.sync = (uint32_t *)(c.ws + 256) + kFp8TileSync;
  a.part = (float *)(c.ws + MOE_WS_FIXED_BYTES);
  if (fp8_tc_ok(a))
    return a.R <= (c.swiglu ? kFp8FewSwiglu : kFp8FewProduct64) * a.E
               ? launch_fp8_few(a, c.swiglu, c.stream)
               : launch_fp8_tc(a, c.swiglu, c.stream);
  return c.swiglu ? run_core<true>(a, c.stream) : run_core<false>(a, c.stream);
}

}  // namespace moe
