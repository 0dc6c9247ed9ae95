// fp8_tc.cu -- routed and dense products over block-scaled e4m3 operands on the
// 5th-generation tensor cores.
//
// A tile is up to MT activation rows of one expert by 256 weight rows (256
// columns of the product; SwiGLU: the gate and up rows of one block of 128
// features).  Per block of 128 along K, tcgen05.mma kind::f8f6f4 (M = 128, N =
// 256, K = 32 four times) forms the unscaled products in one of two TMEM
// accumulators, and the epilogue warps add them, times scale_x * scale_w, to fp32
// sums in registers: the scales change every 128 K, so each accumulator is read
// once per block.  The activation rows sit on the MMA's M side, so that an
// epilogue thread owns one row: its scale product is one scalar per block and
// matrix, a pair of columns costs one packed FMA, and a row's quantisation block
// after SwiGLU is a maximum over the thread's own registers.
//
// Dead rows (tiles of a few rows) cost MMA time but no bytes: at M = 128 the
// tensor cores consume a block's 32 KB of weights in ~512 clocks, HBM delivers an
// SM's share of them in ~1400, so one layout serves decode and prefill.
// Activation rows come by TMA gather (4 rows a request, through perm), so no
// permuted copy of the activations is written.
//
// Warps: 0 weights producer, 1 TMEM owner and MMA issuer, 2 activation producer,
// 3 idle, 4..11 epilogue (warp w reads TMEM lanes 32*(w%4).., columns by half).
//
// Work is split evenly over one CTA per SM: whole tiles in rounds of one per CTA,
// and the tiles of the last, partial round cut along K into equal shares (first in
// every CTA's order).  The shares of a tile meet in the workspace: each CTA writes
// its fp32 sums, the last one to arrive adds all of them in ascending K, so the
// result does not depend on the order of arrival.
#include <cuda.h>
#include <string.h>

#include "fp8_tc.cuh"

namespace moe {
namespace {

constexpr int kTcThreads = 12 * 32;
constexpr int kEpiWarp0 = 4;
constexpr uint32_t kWBytes = 128 * 128;  // one weight box: 128 rows of one K block
constexpr int kMinShare = 4;             // K blocks a CTA takes of a split round, at least
constexpr long long kWaitCycles = 4000000000ll;  // ~2 s
constexpr int kSpin = 1 << 26;
constexpr int kHintNs = 20000;  // try_wait suspend-time hint: waiting warps sleep, not spin
// registers per thread after the split: 128 * 64 + 256 * 216 <= 384 * 168
constexpr int kRegsRole = 64, kRegsEpi = 216;

struct Fp8Maps {
  CUtensorMap x;     // [n_x][K] codes, one row of 128 a box (gathered 4 at a time)
  CUtensorMap w[2];  // [E][N][K] codes, box 128 x 128
};

// ---------------------------------------------------------------- PTX helpers
__device__ __forceinline__ uint32_t s32(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void bar_init(uint64_t *b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(s32(b)), "r"(n));
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(s32(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(s32(b)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool bar_wait(uint64_t *b, uint32_t parity) {
  const long long t0 = clock64();
  for (int i = 0; i < kSpin; ++i) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(s32(b)), "r"(parity), "n"(kHintNs)
        : "memory");
    if (done) return true;
    if (clock64() - t0 > kWaitCycles) return false;
  }
  return false;
}
__device__ __forceinline__ void tma_w(void *dst, const CUtensorMap *map, int k, int n, int e,
                                      uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(s32(dst)),
      "l"(map), "r"(k), "r"(n), "r"(e), "r"(s32(bar))
      : "memory");
}
// four rows of the map's 128-byte boxes to consecutive rows of shared memory
__device__ __forceinline__ void tma_gather4(void *dst, const CUtensorMap *map, int k,
                                            const int (&row)[4], uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(s32(dst)),
      "l"(map), "r"(k), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3]), "r"(s32(bar))
      : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// called by a whole converged warp with uniform operands; one lane issues
__device__ __forceinline__ void tc_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred e, p;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          s32(bar))
      : "memory");
}
// 32 consecutive fp32 columns of this warp's 32 TMEM lanes, no wait
__device__ __forceinline__ void tc_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// waits for the warp's loads; v, the registers of the latest, pass through it so
// that no use of them can move above the wait
__device__ __forceinline__ void tc_wait_ld32(float (&v)[32]) {
#define R4(i) "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3])
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : R4(0), R4(4), R4(8), R4(12), R4(16), R4(20), R4(24), R4(28)::"memory");
#undef R4
}
__device__ __forceinline__ void st_global32(void *p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// shared-memory matrix descriptor: K-major operand, 128-byte swizzle (8-row groups
// of 1024 bytes), version 1
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// instruction descriptor: D f32, A and B e4m3, both K-major, N >> 3 at bit 17, M = 128
__device__ __forceinline__ uint32_t idesc_for(uint32_t n) {
  return (1u << 4) | ((n >> 3) << 17) | (8u << 24);
}

// ---------------------------------------------------------------- work split
// A CTA's work in order: its share [pos, end) of the split tiles' K blocks, then
// whole tiles split, split + G, ...  Every role walks the same list.
struct Seg {
  int tile, kb0, kb1;
};
struct Walk {
  int n_all, split, share, kbs, grid;  // tiles, split tiles, K blocks per CTA, per tile
  int pos, end, next;
  __device__ Walk(int n_all_, int kbs_) : n_all(n_all_), kbs(kbs_), grid(gridDim.x) {
    split = n_all % grid;
    const long long items = (long long)split * kbs;
    share = max((int)((items + grid - 1) / grid), min(kMinShare, kbs));
    pos = (int)min(items, (long long)blockIdx.x * share);
    end = (int)min(items, (long long)pos + share);
    next = split + blockIdx.x;
  }
  __device__ bool take(Seg &s) {
    if (pos < end) {
      s.tile = pos / kbs;
      s.kb0 = pos - s.tile * kbs;
      s.kb1 = min(kbs, s.kb0 + end - pos);
      pos += s.kb1 - s.kb0;
      return true;
    }
    if (next >= n_all) return false;
    s.tile = next;
    s.kb0 = 0;
    s.kb1 = kbs;
    next += grid;
    return true;
  }
  // CTAs that share split tile v
  __device__ int first_cta(int v) const { return (int)((long long)v * kbs / share); }
  __device__ int last_cta(int v) const { return (int)(((long long)(v + 1) * kbs - 1) / share); }
};

// Row r's product over one segment leaves 128 fp32 sums in each of its two
// epilogue threads: acc[0..31] and acc[32..63] are pairs of columns -- of the
// gate and the up block (SwiGLU), or of the two halves of 128 columns.
template <bool SWIGLU, int MT>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_fp8_tc(const Fp8Args a, const __grid_constant__ Fp8Maps maps, const int n_stages,
             const bool vec) {
  pdl_trigger();
  extern __shared__ __align__(1024) uint8_t tsm_raw[];
  uint8_t *tsm = (uint8_t *)(((uintptr_t)tsm_raw + 1023) & ~(uintptr_t)1023);
  constexpr uint32_t kABytes = MT * 128, kStage = kABytes + 2 * kWBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t *ctrl = tsm + (size_t)n_stages * kStage;
  uint64_t *full = (uint64_t *)ctrl;    // [8] operands of a stage landed
  uint64_t *empty = full + 8;           // [8] ... consumed
  uint64_t *d_full = empty + 8;         // [2] accumulator written
  uint64_t *d_empty = d_full + 2;       // [2] ... read
  uint64_t *pair = d_empty + 2;         // [4] the two epilogue warps of a lane quarter
  uint32_t *tmem_holder = (uint32_t *)(pair + 4);
  volatile int *abort_flag = (volatile int *)(tmem_holder + 1);
  volatile int *last_part = (volatile int *)(tmem_holder + 2);  // [4]
  float *ex = (float *)(ctrl + 256);                            // [2][2][128] row maxima
  int *tiles_sm = (int *)(ctrl + 256 + 2048);

  if (tid == 0) {
    for (int i = 0; i < 8; ++i) {
      bar_init(&full[i], 2);
      bar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&d_full[i], 1);
      bar_init(&d_empty[i], 8);
    }
    for (int i = 0; i < 4; ++i) bar_init(&pair[i], 2);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     s32(tmem_holder))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_wait();
  const RowTiles rt = fp8_row_tiles<MT>(a, tiles_sm);
  Walk walk(rt.total * (int)a.n_tiles, (int)a.nbk);
  Seg seg;
  auto give_up = [&]() {
    atomicOr(a.err, kErrTimeout);
    *abort_flag = 1;
  };
  // weight blocks of a tile: SwiGLU one of each matrix, else 2 (1 at the end of N)
  auto halves = [&](const Fp8Tile &t) {
    return SWIGLU || (uint32_t)t.nt * 256 + 128 < a.N ? 2 : 1;
  };

  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRole));
    if (warp == 0 && lane == 0) {
      // ============================ weights
      uint32_t g = 0;
      while (!*abort_flag && walk.take(seg)) {
        const Fp8Tile t = fp8_tile<MT>(a, rt, seg.tile);
        const int nh = halves(t);
        for (int kb = seg.kb0; kb < seg.kb1; ++kb, ++g) {
          const uint32_t s = g % n_stages;
          if (g >= (uint32_t)n_stages && !bar_wait(&empty[s], (g / n_stages - 1) & 1)) {
            give_up();
            break;
          }
          uint8_t *dst = tsm + (size_t)s * kStage + kABytes;
          bar_expect(&full[s], nh * kWBytes);
          if (SWIGLU) {
            tma_w(dst, &maps.w[0], kb * 128, t.nt * 128, t.e, &full[s]);
            tma_w(dst + kWBytes, &maps.w[1], kb * 128, t.nt * 128, t.e, &full[s]);
          } else {
            for (int h = 0; h < nh; ++h)
              tma_w(dst + h * kWBytes, &maps.w[0], kb * 128, t.nt * 256 + 128 * h, t.e, &full[s]);
          }
        }
      }
      // the stages still in use: leave with no copy in flight
      for (uint32_t i = g > (uint32_t)n_stages ? g - n_stages : 0; i < g; ++i)
        if (!bar_wait(*abort_flag ? &full[i % n_stages] : &empty[i % n_stages],
                      (i / n_stages) & 1))
          give_up();
    } else if (warp == 1) {
      // ============================ MMA issuer
      uint32_t g = 0;
      while (!*abort_flag && walk.take(seg)) {
        const Fp8Tile t = fp8_tile<MT>(a, rt, seg.tile);
        const uint32_t idesc = idesc_for(128 * halves(t));
        for (int kb = seg.kb0; kb < seg.kb1; ++kb, ++g) {
          const uint32_t s = g % n_stages, b = g & 1;
          if ((g >= 2 && !bar_wait(&d_empty[b], (g / 2 - 1) & 1)) ||
              !bar_wait(&full[s], (g / n_stages) & 1)) {
            give_up();
            break;
          }
          tc_fence_after();
          __syncwarp();
          const uint64_t ad = sw128_desc(s32(tsm + (size_t)s * kStage));
          const uint64_t bd = sw128_desc(s32(tsm + (size_t)s * kStage + kABytes));
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 32 bytes along K: 2 in the descriptor's units
            tc_mma(tmem + b * 256, ad + 2 * k, bd + 2 * k, idesc, k > 0);
          tc_commit(&empty[s]);
          tc_commit(&d_full[b]);
        }
      }
    } else if (warp == 2) {
      // ============================ activations: lane l gathers rows 4l..4l+3
      uint32_t g = 0;
      while (!*abort_flag && walk.take(seg)) {
        const Fp8Tile t = fp8_tile<MT>(a, rt, seg.tile);
        const int groups = (t.rows + 3) / 4;
        int row[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // rows past the end repeat the last one; a bad one reads row 0 (flagged)
          const int r = min(4 * lane + i, t.rows - 1);
          row[i] = max(0, fp8_x_row(a, t.row0 + r));
        }
        for (int kb = seg.kb0; kb < seg.kb1; ++kb, ++g) {
          const uint32_t s = g % n_stages;
          if (g >= (uint32_t)n_stages && !bar_wait(&empty[s], (g / n_stages - 1) & 1)) {
            give_up();
            break;
          }
          if (lane == 0) bar_expect(&full[s], groups * 512);
          __syncwarp();
          if (lane < groups)
            tma_gather4(tsm + (size_t)s * kStage + lane * 512, &maps.x, kb * 128, row, &full[s]);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    // ============================ epilogue
    const int ew = warp - kEpiWarp0, half = ew >> 2, quarter = warp & 3;
    const int m = quarter * 32 + lane;  // row of the tile, TMEM lane
    const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
    uint32_t g = 0, npair = 0;  // accumulators, and meetings of the pair, so far
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) bar_arrive(&pair[quarter]);
      const bool ok = bar_wait(&pair[quarter], npair++ & 1);
      if (!ok) give_up();
      return ok;
    };
    uint32_t n_ex = 0;
    while (!*abort_flag && walk.take(seg)) {
      const Fp8Tile t = fp8_tile<MT>(a, rt, seg.tile);
      const bool warp_live = quarter * 32 < t.rows && (SWIGLU || half < halves(t));
      const bool live = warp_live && m < t.rows;
      const float *xs = a.xs, *wa = a.wsc[0], *wb = a.wsc[0];
      if (warp_live) {
        const int r = t.row0 + min(m, t.rows - 1);
        xs = a.xs + (size_t)max(0, fp8_x_row(a, r)) * a.nbk;
        const size_t blk = SWIGLU ? t.nt : 2 * t.nt + half;
        wa = a.wsc[0] + ((size_t)t.e * a.nbn + blk) * a.nbk;
        wb = SWIGLU ? a.wsc[1] + ((size_t)t.e * a.nbn + blk) * a.nbk : wa;
      }
      float2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.0f, 0.0f);
      float sx = 0.0f, sa = 0.0f, sb = 0.0f;
      if (warp_live) sx = xs[seg.kb0], sa = wa[seg.kb0], sb = wb[seg.kb0];
      bool ok = true;
      for (int kb = seg.kb0; kb < seg.kb1; ++kb, ++g) {
        const uint32_t b = g & 1;
        if (!bar_wait(&d_full[b], (g / 2) & 1)) {
          give_up();
          ok = false;
          break;
        }
        if (warp_live) {
          tc_fence_after();
          const float s0 = sx * sa, s1 = sx * sb;
          // the next block's scales, on the way while this one is added
          const int kn = min(kb + 1, seg.kb1 - 1);
          sx = xs[kn], sa = wa[kn], sb = wb[kn];
          const uint32_t base = lane_addr + b * 256;
          const uint32_t c0 = SWIGLU ? 64 * half : 128 * half, c1 = SWIGLU ? 128 + 64 * half
                                                                           : 128 * half + 64;
          float v[2][32];
          tc_ld32(base + c0, v[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tc_wait_ld32(v[c & 1]);
            if (c < 3) tc_ld32(base + (c < 1 ? c0 + 32 : c1 + 32 * (c - 1)), v[(c + 1) & 1]);
            const float s = c < 2 ? s0 : s1;
            const float2 s2 = make_float2(s, s);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              acc[16 * c + i] = __ffma2_rn(make_float2(v[c & 1][2 * i], v[c & 1][2 * i + 1]), s2,
                                           acc[16 * c + i]);
          }
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&d_empty[b]);
      }
      if (!ok) break;
      // ---- a share of a tile: the last of its CTAs adds up all shares
      if (seg.kb1 - seg.kb0 < (int)a.nbk) {
        if (quarter * 32 >= t.rows) continue;  // both warps of the pair
        const int c0 = walk.first_cta(seg.tile), n = walk.last_cta(seg.tile) - c0 + 1;
        // part of CTA c: its second slot if it starts the tile, its first otherwise
        auto part = [&](int c) {
          return (float4 *)(a.part + (size_t)(2 * c + (c == c0)) * a.part_stride) +
                 (size_t)(quarter * 2 + half) * 1024 + lane;
        };
        float4 *mine = part((int)blockIdx.x);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          __stcg(mine + 32 * i,
                 make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y));
        __threadfence();
        if (!meet()) break;
        uint32_t *count = a.sync + 4 * seg.tile + quarter;
        if (half == 0 && lane == 0) {
          __threadfence();
          const bool last = atomicAdd(count, 1u) == (uint32_t)n - 1;
          if (last) atomicExch(count, 0u);
          last_part[quarter] = last;
        }
        if (!meet()) break;
        if (!last_part[quarter]) continue;
        __threadfence();
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.0f, 0.0f);
        for (int p = 0; p < n; ++p) {
          const float4 *src = part(c0 + p);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float4 v = __ldcg(src + 32 * i);
            acc[2 * i].x += v.x;
            acc[2 * i].y += v.y;
            acc[2 * i + 1].x += v.z;
            acc[2 * i + 1].y += v.w;
          }
        }
      }
      // ---- outputs
      const int r = t.row0 + m;
      if (!SWIGLU) {
        if (!live) continue;
        const uint32_t n0 = (uint32_t)t.nt * 256 + 128 * half;
        if (vec) {
          if (a.odt == MOE_DT_F32) {
            float *dst = (float *)a.out + (size_t)r * a.ld + n0;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (n0 + 8 * i < a.N) {
                const uint32_t w[8] = {
                    __float_as_uint(acc[4 * i].x),     __float_as_uint(acc[4 * i].y),
                    __float_as_uint(acc[4 * i + 1].x), __float_as_uint(acc[4 * i + 1].y),
                    __float_as_uint(acc[4 * i + 2].x), __float_as_uint(acc[4 * i + 2].y),
                    __float_as_uint(acc[4 * i + 3].x), __float_as_uint(acc[4 * i + 3].y)};
                st_global32(dst + 8 * i, w);
              }
          } else {
            uint16_t *dst = (uint16_t *)a.out + (size_t)r * a.ld + n0;
            const bool bf = a.odt == MOE_DT_BF16;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (n0 + 16 * i < a.N) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  w[j] = bf ? pack2<MOE_DT_BF16>(acc[8 * i + j].x, acc[8 * i + j].y)
                            : pack2<MOE_DT_F16>(acc[8 * i + j].x, acc[8 * i + j].y);
                st_global32(dst + 16 * i, w);
              }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            if (n0 + 2 * i < a.N) fp8_store(a, r, n0 + 2 * i, acc[i].x);
            if (n0 + 2 * i + 1 < a.N) fp8_store(a, r, n0 + 2 * i + 1, acc[i].y);
          }
        }
      } else {
        if (!warp_live) continue;
        // h of this thread's 64 features (past N: g = u = 0, h = 0), and the row's
        // maximum with the partner thread's
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          acc[i].x = fp8_swiglu_value(acc[i].x, acc[32 + i].x);
          acc[i].y = fp8_swiglu_value(acc[i].y, acc[32 + i].y);
          amax = fmaxf(amax, fmaxf(fabsf(acc[i].x), fabsf(acc[i].y)));
        }
        float *e = ex + (n_ex++ & 1) * 256;
        e[128 * half + m] = amax;
        if (!meet()) break;
        amax = fmaxf(amax, e[128 * (half ^ 1) + m]);
        float sc, inv;
        fp8_block_scale(amax, sc, inv);
        if (!live) continue;
        if (half == 0) a.hs[(size_t)r * a.nbn + t.nt] = sc;
        const uint32_t n0 = (uint32_t)t.nt * 128 + 64 * half;
        uint8_t *dst = (uint8_t *)a.out + (size_t)r * a.N + n0;
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = e4m3x4(acc[2 * i].x * inv, acc[2 * i].y * inv, acc[2 * i + 1].x * inv,
                        acc[2 * i + 1].y * inv);
        if (vec) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (n0 + 32 * i < a.N) {
              const uint32_t q[8] = {w[8 * i],     w[8 * i + 1], w[8 * i + 2], w[8 * i + 3],
                                     w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]};
              st_global32(dst + 32 * i, q);
            }
        } else {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (n0 + i < a.N) dst[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ---------------------------------------------------------------- host
typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
  static EncodeTiled fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeTiled)p;
  }();
  return fn;
}

// byte matrices [d2][d1][K], box 128 bytes of box_rows rows, 128-byte swizzle
bool byte_map(CUtensorMap *m, const void *base, uint64_t K, uint64_t d1, uint64_t d2, int dims,
              uint32_t box_rows) {
  const cuuint64_t size[3] = {K, d1, d2};
  const cuuint64_t stride[2] = {K, K * d1};
  const cuuint32_t box[3] = {128, box_rows, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, dims, const_cast<void *>(base), size, stride,
                     box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kSmemLimit = 232448;

template <bool SWIGLU, int MT>
cudaError_t run_tc(Fp8Args &a, const Fp8Maps &maps, int sms, bool vec, cudaStream_t stream) {
  auto kern = k_fp8_tc<SWIGLU, MT>;
  const size_t stage = MT * 128 + 2 * (size_t)kWBytes;
  const size_t rest = 1024 + 256 + 2048 + fp8_tiles_smem(a.E);
  int ns = (int)((kSmemLimit - rest) / stage);
  if (ns > 8) ns = 8;
  const size_t smem = rest + ns * stage;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_k(kern, sms, kTcThreads, smem, stream, true, a, maps, ns, vec);
}

}  // namespace

bool fp8_tc_ok(const Fp8Args &a) {
  auto a16 = [](const void *p) { return ((uintptr_t)p & 15) == 0; };
  return a.K % 16 == 0 && a16(a.xq) && a16(a.wq[0]) && a16(a.wq[1]) && encode_fn() != nullptr;
}

size_t fp8_tc_ws(uint32_t rows) {
  // two parts a CTA, each 128 sums of fp32 in 64 threads per 32 rows
  const size_t quarters = ((rows < 128 ? rows : 128) + 31) / 32;
  return (size_t)fp8_ctas() * 2 * quarters * 32768;
}

cudaError_t launch_fp8_tc(Fp8Args &a, bool swiglu, cudaStream_t stream) {
  const int sms = fp8_ctas();
  const uint32_t quarters = ((a.R < 128 ? a.R : 128) + 31) / 32;
  a.part_stride = (size_t)quarters * 8192;
  a.n_tiles = swiglu ? a.nbn : (a.nbn + 1) / 2;
  Fp8Maps maps;
  memset(&maps, 0, sizeof maps);
  if (!byte_map(&maps.x, a.xq, a.K, a.n_x, 1, 2, 1) ||
      !byte_map(&maps.w[0], a.wq[0], a.K, a.N, a.E, 3, 128) ||
      (swiglu && !byte_map(&maps.w[1], a.wq[1], a.K, a.N, a.E, 3, 128)))
    return cudaErrorInvalidValue;
  if (!swiglu) maps.w[1] = maps.w[0];
  // 32-byte stores: whole groups of 32 bytes inside every row
  const uint32_t group = 32 / (swiglu ? 1 : (uint32_t)dtype_size(a.odt));
  const bool vec = ((uintptr_t)a.out & 31) == 0 && a.N % group == 0 && a.ld % group == 0;
  if (swiglu)
    return a.R <= 32 * a.E ? run_tc<true, 32>(a, maps, sms, vec, stream)
                           : run_tc<true, 128>(a, maps, sms, vec, stream);
  return a.R <= 32 * a.E ? run_tc<false, 32>(a, maps, sms, vec, stream)
                         : run_tc<false, 128>(a, maps, sms, vec, stream);
}

}  // namespace moe
