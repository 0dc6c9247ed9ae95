// fp8_tiles.cuh -- the row tiles of a routed product: which expert and which of
// its rows a tile number names, from off[] alone, worked out by every CTA for
// itself (E+1 loads and one block scan, no plan kernel before the product).
#pragma once

#include "fp8_common.cuh"

namespace moe {

constexpr uint32_t kFp8MaxExperts = 1024;

// arguments shared by the product kernels
struct Fp8Args {
  uint32_t E, N, K, nbn, nbk;  // nbn, nbk: blocks of 128 along N and K
  uint32_t n_x, R, top_k;      // activation rows, output rows
  const uint8_t *xq;
  const float *xs;
  const int32_t *off, *perm;
  const uint8_t *wq[2];
  const float *wsc[2];
  void *out;    // product output, or h codes
  size_t ld;
  float *hs;
  int odt;
  uint32_t n_tiles;    // column tiles of an expert
  uint32_t *err, *sync;
  float *part;         // partial sums of split tiles
  size_t part_stride;  // floats per part
};

// activation row of output row r; -1 (flagged) if perm names none
__device__ __forceinline__ int fp8_x_row(const Fp8Args &a, int r) {
  const uint32_t x = a.perm ? (uint32_t)a.perm[r] / a.top_k : (uint32_t)r;
  if (x < a.n_x) return (int)x;
  atomicOr(a.err, kErrBadIndex);
  return -1;
}

// off[] and the exclusive prefix of the row tiles (MT rows each) in shared
// memory; total is 0 where off is not ascending within [0, R] (flagged)
struct RowTiles {
  const int *off, *tile;  // [E+1] each
  int total;
};

// called by all threads (a multiple of 32, at most 1024); sm: 2(E+1) + 34 ints
template <int MT>
__device__ __forceinline__ RowTiles fp8_row_tiles(const Fp8Args &a, int *sm) {
  int *s_off = sm, *s_tile = sm + (a.E + 1), *wsum = s_tile + (a.E + 1), *flag = wsum + 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x;
  if (tid == 0) *flag = 0;
  for (int e = tid; e <= (int)a.E; e += nthr)
    s_off[e] = a.off ? a.off[e] : e == 0 ? 0 : (int)a.R;
  __syncthreads();
  const int per = ((int)a.E + nthr - 1) / nthr;
  const int b = min((int)a.E, tid * per), e1 = min((int)a.E, b + per);
  int sum = 0;
  for (int e = b; e < e1; ++e) {
    const int rows = s_off[e + 1] - s_off[e];
    if (rows < 0 || s_off[e] < 0 || s_off[e + 1] > (int)a.R) *flag = 1;
    sum += (max(rows, 0) + MT - 1) / MT;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int run = incl - sum, total = 0;
  for (int w = 0; w < nthr / 32; ++w) {
    if (w < warp) run += wsum[w];
    total += wsum[w];
  }
  for (int e = b; e < e1; ++e) {
    s_tile[e] = run;
    run += (max(s_off[e + 1] - s_off[e], 0) + MT - 1) / MT;
  }
  if (tid == 0) s_tile[a.E] = total;
  const bool bad = *flag != 0;
  if (bad && tid == 0) atomicOr(a.err, kErrBadOffsets);
  __syncthreads();
  RowTiles t;
  t.off = s_off;
  t.tile = s_tile;
  t.total = bad ? 0 : total;
  return t;
}

struct Fp8Tile {
  int e, row0, rows, nt;  // expert, first output row, live rows, column tile
};

// tile v of total * n_tiles: experts in order, an expert's column tiles one
// after another, its row tiles innermost (they share the weights)
template <int MT>
__device__ __forceinline__ Fp8Tile fp8_tile(const Fp8Args &a, const RowTiles &rt, int v) {
  // expert e's tiles are [tile[e] * n_tiles, tile[e+1] * n_tiles)
  const int q = v / (int)a.n_tiles;
  int lo = 0, hi = (int)a.E;  // largest e with tile[e] <= q (experts without rows share a prefix)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (rt.tile[mid] <= q) lo = mid; else hi = mid;
  }
  const int mt = rt.tile[lo + 1] - rt.tile[lo];
  const int local = v - rt.tile[lo] * (int)a.n_tiles;
  Fp8Tile t;
  t.e = lo;
  t.nt = local / mt;
  const int m = local - t.nt * mt;
  t.row0 = rt.off[lo] + m * MT;
  t.rows = min(MT, rt.off[lo + 1] - t.row0);
  return t;
}

inline size_t fp8_tiles_smem(uint32_t E) { return 4 * (2 * ((size_t)E + 1) + 34); }

// store one output value of the product
__device__ __forceinline__ void fp8_store(const Fp8Args &a, int r, uint32_t n, float v) {
  const size_t i = (size_t)r * a.ld + n;
  if (a.odt == MOE_DT_F32) ((float *)a.out)[i] = v;
  else if (a.odt == MOE_DT_BF16) ((__nv_bfloat16 *)a.out)[i] = __float2bfloat16_rn(v);
  else ((__half *)a.out)[i] = __float2half_rn(v);
}

// h = g / (1 + e^-g) * u
__device__ __forceinline__ float fp8_swiglu_value(float g, float u) {
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

}  // namespace moe
