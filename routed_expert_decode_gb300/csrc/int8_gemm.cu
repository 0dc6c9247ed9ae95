// int8_gemm.cu -- routed and dense products over int8 operands with a scale per weight
// row and per activation row, on CUDA cores: the kernel for operands that tensor copies
// cannot take (a reduction length that is not a multiple of 16, code planes that are
// not 16-byte aligned).  Sums are exact, in 32-bit integers.
#include "int8.cuh"

namespace moe {
namespace {

constexpr int kCoreM = 32, kCoreN = 128;  // rows and columns of a tile
constexpr int kCoreThreads = 256;
constexpr int kSlab = 128;                 // codes of K staged at a time
constexpr int kPitch = kSlab / 4 + 1;      // words of a staged row: columns in distinct banks

// Thread (ty, tx) holds rows ty + 8i and columns tx + 32j; the codes of a slab of K are
// staged as words of four and multiplied four at a time.
template <bool SWIGLU>
__global__ void __launch_bounds__(kCoreThreads) k_int8_core(const Fp8Args a) {
  pdl_trigger();
  pdl_wait();
  constexpr int NM = SWIGLU ? 2 : 1;
  extern __shared__ __align__(16) uint8_t csm[];
  uint32_t *sx = (uint32_t *)csm;           // [kCoreM][kPitch]
  uint32_t *sw = sx + kCoreM * kPitch;      // [NM][kCoreN][kPitch]
  int *tiles_sm = (int *)(sw + NM * kCoreN * kPitch);
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
    int acc[NM][4][4];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][i][j] = 0;
    for (uint32_t k0 = 0; k0 < a.K; k0 += kSlab) {
      auto word = [&](const uint8_t *row) {  // codes 4 tx .. of the slab, 0 past K
        uint32_t w = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (k0 + 4 * tx + b < a.K) w |= (uint32_t)row[k0 + 4 * tx + b] << (8 * b);
        return w;
      };
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sx[(ty + 8 * i) * kPitch + tx] = xrow[i] >= 0 ? word(a.xq + (size_t)xrow[i] * a.K) : 0;
#pragma unroll
      for (int m = 0; m < NM; ++m)
        for (int n = ty; n < kCoreN; n += 8)
          sw[(m * kCoreN + n) * kPitch + tx] =
              n0 + n < a.N ? word(a.wq[m] + ((size_t)t.e * a.N + n0 + n) * a.K) : 0;
      __syncthreads();
#pragma unroll 4
      for (int q = 0; q < kSlab / 4; ++q) {
        int xv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) xv[i] = (int)sx[(ty + 8 * i) * kPitch + q];
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int wv = (int)sw[(m * kCoreN + tx + 32 * j) * kPitch + q];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][i][j] = __dp4a(xv[i], wv, acc[m][i][j]);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (ty + 8 * i >= t.rows) continue;
      const int r = t.row0 + ty + 8 * i;
      const float xs = xrow[i] >= 0 ? a.xs[xrow[i]] : 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t n = n0 + tx + 32 * j;
        if (n >= a.N) continue;
        const size_t ch = (size_t)t.e * a.N + n;
        float y = (float)acc[0][i][j] * (xs * a.wsc[0][ch]);
        if (SWIGLU) y = fp8_swiglu_value(y, (float)acc[NM - 1][i][j] * (xs * a.wsc[NM - 1][ch]));
        fp8_store(a, r, n, y);
      }
    }
  }
}

template <bool SWIGLU>
cudaError_t run_core(Fp8Args &a, cudaStream_t stream) {
  auto kern = k_int8_core<SWIGLU>;
  fp8_set_tiles(a, fp8_blocks(a.N), 1);
  const size_t smem =
      4 * (size_t)((kCoreM + (SWIGLU ? 2 : 1) * kCoreN) * kPitch) + fp8_tiles_smem(a.E);
  static std::atomic<bool> done[kMaxDevices];
  const cudaError_t e = allow_smem(kern, done);
  if (e != cudaSuccess) return e;
  return launch_k(kern, 4 * fp8_ctas(), kCoreThreads, smem, stream, true, a);
}

// The stream kernel for few rows takes calls whose rows have about an expert each (or no more
// than four in all) and whose activations fit a CTA's shared memory; the tensor-core kernel
// those whose experts have several.  Top 8 of 256, d 6144, f 2048, us, stream and tensor-core:
//   tokens           1         2         4         8        16        24
//   gate/up    36   43   60   70  104  114  180  201  275  298  376  391
//   down       21   26   36   39   60   63  100  108              118  115 (K 1024)
// 64 and 128 rows of 16 experts (gate/up): 77 and 72, 120 and 79; 16 of 4: 28 and 24; one
// expert, K 6144: 4 rows 11.2 and 14.1, 8 rows (gate/up) 12 and 15, 12 rows 19 and 16; K 1024,
// 8 rows: 12 and 7.
bool few_rows(const Fp8Args &a) {
  return 2ull * a.R <= (a.E > 8 ? a.E : 8) && (uint64_t)a.n_x * a.K <= 200 * 1024 &&
         (uint64_t)a.R * (a.N / 2 + 1) < (1ull << 31);  // its units are numbered in 31 bits
}

}  // namespace

size_t int8_gemm_ws() { return MOE_WS_FIXED_BYTES + int8_tc_ws(); }

cudaError_t launch_int8_gemm(const Int8Call &c) {
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
  a.odt = c.odt;
  a.err = (uint32_t *)c.ws;
  a.sync = (uint32_t *)(c.ws + 256) + kFp8TileSync;
  a.part = (float *)(c.ws + MOE_WS_FIXED_BYTES);
  if (int8_tc_ok(a))
    return few_rows(a) ? launch_int8_few(a, c.swiglu, c.stream)
                       : launch_int8_tc(a, c.swiglu, c.stream);
  return c.swiglu ? run_core<true>(a, c.stream) : run_core<false>(a, c.stream);
}

}  // namespace moe
