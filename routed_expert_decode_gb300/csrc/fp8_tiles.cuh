// fp8_tiles.cuh -- the row tiles of a routed product: which expert and which of
// its rows a tile number names, from off[] alone, worked out by every CTA for
// itself (E+1 loads and one block scan, no plan kernel before the product).
#pragma once

#include "fp8_common.cuh"

namespace moe {

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
  uint32_t n_tiles, n_tiles_inv;  // column tiles of an expert, floor((2^32 - 1) / that)
  uint32_t workers_inv;           // the same of the CTAs that share the tiles
  uint32_t *err, *sync;
  float *part;         // partial sums of split tiles
  size_t part_stride;  // floats per part
};

// Before the wait for the stream's earlier work: the arguments into the constant
// cache (a launch's are always cold, and the first uses come one after another)
// and the routing arrays' lines on their way to L2 (a prefetch there reads nothing).
__device__ __forceinline__ void fp8_warm(const Fp8Args &a) {
  asm volatile("" ::"r"(a.E), "r"(a.N), "r"(a.nbn), "r"(a.nbk), "r"(a.R), "r"(a.top_k), "l"(a.xq),
               "l"(a.xs), "l"(a.off), "l"(a.perm), "l"(a.wsc[0]), "l"(a.wsc[1]), "l"(a.out),
               "l"(a.hs), "r"(a.n_tiles), "r"(a.n_tiles_inv), "r"(a.workers_inv), "l"(a.err), "l"(a.sync),
               "l"(a.part));
  auto prefetch = [](const int32_t *p, uint32_t n) {
    const uint32_t i = threadIdx.x * 32;
    if (p && i < n) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i));
  };
  prefetch(a.off, a.E + 1);
  prefetch(a.perm, a.R);
}

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

// called by all threads; sm: 2(E+1) + 1 ints.  One warp does it, a run of experts a
// lane, behind a single block barrier: it is on every call's critical path.
template <int MT>
__device__ __forceinline__ RowTiles fp8_row_tiles(const Fp8Args &a, int *sm) {
  int *s_off = sm, *s_tile = sm + (a.E + 1), *s_total = s_tile + (a.E + 1);
  const int E = (int)a.E, R = (int)a.R;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int per = (E + 31) / 32, b = min(E, lane * per), e1 = min(E, b + per);
    auto off = [&](int e) { return a.off ? a.off[e] : e == 0 ? 0 : R; };
    auto warp_scan = [&](int v) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      return v;
    };
    int at = off(b), tiles = 0, incl;
    bool bad = at < 0 || at > R;
    if (per <= 8) {
      int next[8], before[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) next[i] = b + i < e1 ? off(b + i + 1) : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        before[i] = tiles;
        if (b + i < e1) {
          s_off[b + i] = at;
          bad |= next[i] < at || next[i] > R;
          tiles += (max(next[i] - at, 0) + MT - 1) / MT;
          at = next[i];
        }
      }
      incl = warp_scan(tiles);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (b + i < e1) s_tile[b + i] = incl - tiles + before[i];
    } else {
#pragma unroll 8
      for (int e = b; e < e1; ++e) {
        const int next = off(e + 1);
        s_off[e] = at;
        s_tile[e] = tiles;  // within the lane's run so far
        bad |= next < at || next > R;
        tiles += (max(next - at, 0) + MT - 1) / MT;
        at = next;
      }
      incl = warp_scan(tiles);
      for (int e = b; e < e1; ++e) s_tile[e] += incl - tiles;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 31) {
      s_off[E] = at;
      s_tile[E] = incl;
      *s_total = bad ? 0 : incl;
      if (bad) atomicOr(a.err, kErrBadOffsets);
    }
  }
  __syncthreads();
  RowTiles t;
  t.off = s_off;
  t.tile = s_tile;
  t.total = *s_total;
  return t;
}

struct Fp8Tile {
  int e, row0, rows, nt;  // expert, first output row, live rows, column tile
};

// By a whole warp: tile v of total * n_tiles: experts in order, an expert's column tiles one
// after another, its row tiles innermost (they share the weights)
template <int MT>
__device__ __forceinline__ Fp8Tile fp8_tile(const Fp8Args &a, const RowTiles &rt, int v) {
  // expert e's tiles are [tile[e] * n_tiles, tile[e+1] * n_tiles)
  const int q = (int)quotient((uint32_t)v, a.n_tiles, a.n_tiles_inv);
  // the largest e with tile[e] <= q (experts without rows share a prefix): a run of
  // experts a lane, then a lane an expert of that run
  const int lane = threadIdx.x & 31, E = (int)a.E, per = (E + 31) >> 5;
  const int first = lane * per;
  const int run = __popc(__ballot_sync(0xffffffffu, first < E && rt.tile[min(first, E)] <= q)) - 1;
  const int e = run * per + lane;
  const int lo = run * per - 1 +
                 __popc(__ballot_sync(0xffffffffu, lane < per && e < E && rt.tile[min(e, E)] <= q));
  const int mt = rt.tile[lo + 1] - rt.tile[lo];
  const int local = v - rt.tile[lo] * (int)a.n_tiles;
  Fp8Tile t;
  t.e = lo;
  t.nt = mt == 1 ? local : local / mt;
  const int m = local - t.nt * mt;
  t.row0 = rt.off[lo] + m * MT;
  t.rows = min(MT, rt.off[lo + 1] - t.row0);
  return t;
}

inline size_t fp8_tiles_smem(uint32_t E) { return 4 * (2 * ((size_t)E + 1) + 2); }

inline void fp8_set_tiles(Fp8Args &a, uint32_t n_tiles, uint32_t workers) {
  a.n_tiles = n_tiles;
  a.n_tiles_inv = 0xffffffffu / n_tiles;
  a.workers_inv = 0xffffffffu / workers;
}

// store one output value of the product
__device__ __forceinline__ void fp8_store(const Fp8Args &a, int r, uint32_t n, float v) {
  const size_t i = (size_t)r * a.ld + n;
  if (a.odt == MOE_DT_F32) ((float *)a.out)[i] = v;
  else if (a.odt == MOE_DT_BF16) ((__nv_bfloat16 *)a.out)[i] = __float2bfloat16_rn(v);
  else ((__half *)a.out)[i] = __float2half_rn(v);
}

// h = g / (1 + e^-g) * u, with the special function unit's 2^x and 1 / x (2 ulp each).
// Its 1 / x of more than 2^126 (g of -87.4 to -88.7) would be a subnormal, which it
// flushes to 0: a quarter of the divisor never is that large, and a quarter of both
// sides is the same quotient.  A flushed e^-g is nothing beside 1.
__device__ __forceinline__ float fp8_swiglu_value(float g, float u) {
  constexpr float kLog2E = 1.4426950408889634f;
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-kLog2E * g));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fmaf_rn(e, 0.25f, 0.25f)));
  return 0.25f * g * r * u;
}

}  // namespace moe
