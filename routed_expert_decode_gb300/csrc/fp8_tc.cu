// fp8_tc.cu -- routed and dense products over block-scaled e4m3 operands on the
// 5th-generation tensor cores.
//
// A tile is a run of activation rows of one expert by NH blocks of 128 weight rows
// (NH = 2: 256 columns of the product, or the gate and up rows of one block of 128
// features).  Per block of 128 along K, tcgen05.mma kind::f8f6f4 (M = 128 rows a
// CTA, K = 32 four times) forms the unscaled products in one of two TMEM
// accumulators, and the epilogue warps add them, times scale_x * scale_w, to fp32
// sums in registers: the scales change every 128 K, so each accumulator is read
// once per block.  The activation rows sit on the MMA's M side, so that an
// epilogue thread owns one row: its scale product is one scalar per block and
// matrix, a pair of columns costs one packed FMA, and a row's quantisation block
// after SwiGLU is a maximum over two threads' registers.
//
// Dead rows (tiles of a few rows) cost MMA time but no bytes: at M = 128 the
// tensor cores consume a block's 32 KB of weights in ~512 clocks, HBM delivers an
// SM's share of them in ~1400, so one layout serves decode and prefill.
// Routed activation rows are copied by 16-byte cp.async through perm into the
// swizzled layout, so no permuted copy of the activations is written (TMA's
// gather of 4 rows a request took ~78 clocks a request, 2500 a tile of 128 rows);
// rows in order come by one TMA box.
//
// Many rows (CG = 2): a pair of CTAs works on 256 rows with cta_group::2, each SM
// holding its own 128 rows and one of the two weight blocks, so that an SM takes in
// 32 KB a block instead of 48 (an SM's share of L2's bandwidth is ~64 bytes a
// clock, 768 clocks for 48 KB, against the MMA's 512).
//
// Warps: 0 weights producer, 1 TMEM owner and MMA issuer (in the pair's second
// CTA: it passes on that its activations have landed), 2 and 3 activations, 4..11
// epilogue (warp w reads TMEM lanes 32*(w%4).., columns by half).
//
// Work goes out over one CTA (pair) per SM (pair): whole tiles in rounds, and the
// tiles of the last, partial round cut along K into equal shares where whole tiles
// would leave too many SMs idle (first in every CTA's order).  The shares of a
// tile meet in the workspace: each CTA writes its fp32 sums, the last one to
// arrive adds all of them in ascending K, so the result does not depend on the
// order of arrival.
#include <string.h>

#include "fp8_tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kTcThreads = 12 * 32;
constexpr int kEpiWarp0 = 4;
// registers per thread after the split: 128 * 56 + 256 * 224 = 384 * 168, the launch's
constexpr int kRegsRole = 56, kRegsEpi = 224;


// A row's product over one segment leaves up to 128 fp32 sums in each of its two
// epilogue threads: acc[0..31] and acc[32..63] are pairs of columns -- of the
// gate and the up block (SwiGLU), or of a block's two halves.
template <bool SWIGLU, int MT, int NH, int CG>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_fp8_tc(const Fp8Args a, const __grid_constant__ Fp8Maps maps, const uint32_t n_stages,
             const int split_below, const bool vec) {
  static_assert((!SWIGLU || NH == 2) && (CG == 1 || (MT == 128 && NH == 2)), "tile shapes");
  pdl_trigger();
  extern __shared__ __align__(1024) uint8_t tsm_raw[];
  uint8_t *tsm = (uint8_t *)(((uintptr_t)tsm_raw + 1023) & ~(uintptr_t)1023);
  constexpr int kRows = MT * CG;                 // rows of a tile
  constexpr uint32_t kABytes = MT * 128;         // this CTA's activations of a stage
  constexpr uint32_t kWStage = NH / CG * kWBytes;  // its weights
  constexpr uint32_t kStage = kABytes + kWStage;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = CG == 2 ? (int)(blockIdx.x & 1) : 0;  // CTA of the pair
  uint8_t *ctrl = tsm + n_stages * kStage;
  uint64_t *full = (uint64_t *)ctrl;     // [kMaxStages] operands of a stage landed
  uint64_t *empty = full + kMaxStages;   // [kMaxStages] ... consumed
  uint64_t *landed = empty + kMaxStages;  // [kMaxStages] second CTA: its activations landed
  uint64_t *d_full = landed + kMaxStages;  // [2] accumulator written
  uint64_t *d_empty = d_full + 2;        // [2] ... read
  uint64_t *pair = d_empty + 2;          // [4] the two epilogue warps of a lane quarter
  uint64_t *drain = pair + 4;            // the MMAs of an aborted call
  uint32_t *tmem_holder = (uint32_t *)(drain + 1);
  volatile int *abort_flag = (volatile int *)(tmem_holder + 1);
  volatile int *last_part = (volatile int *)(tmem_holder + 2);  // [4]
  float *ex = (float *)(ctrl + 512);                            // [2][2][128] row maxima
  int *tiles_sm = (int *)(ctrl + 512 + 2048);
  const bool gather = a.perm != nullptr;

  if (tid == 32) {
    prefetch_map(&maps.w[0]);
    prefetch_map(&maps.w[1]);
    if (!gather) prefetch_map(&maps.x);
  }
  if (tid == 0) {
    // arrivals on `full`: the weights' producer (with all bytes that tensor copies
    // bring), and the 64 activation threads and the second CTA's forwarder (gather)
    const uint32_t n_full = gather ? 1 + 64 + (CG - 1) : 1;
    for (int i = 0; i < kMaxStages; ++i) {
      bar_init(&full[i], n_full);
      bar_init(&empty[i], 1);
      bar_init(&landed[i], 64);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&d_full[i], 1);
      bar_init(&d_empty[i], 8 * CG);
    }
    for (int i = 0; i < 4; ++i) bar_init(&pair[i], 2);
    bar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    if (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                       s32(tmem_holder))
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                       s32(tmem_holder))
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();  // both CTAs' barriers are set up
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  fp8_warm(a);
  pdl_wait();
  const RowTiles rt = fp8_row_tiles<kRows>(a, tiles_sm);
  const int worker = (int)blockIdx.x / CG;
  Walk walk(rt.total * (int)a.n_tiles, a, worker, (int)gridDim.x / CG, split_below);
  Seg seg;
  const Guard guard{a.err, abort_flag};
  // this CTA's share of a tile: rows from row0 on
  auto my_tile = [&](int v) {
    Fp8Tile t = fp8_tile<kRows>(a, rt, v);
    t.row0 += MT * rank;
    t.rows = max(0, min(MT, t.rows - MT * rank));
    return t;
  };
  // weight blocks that a tile has: the last of an odd number stands alone
  auto blocks_of = [&](const Fp8Tile &t) {
    return SWIGLU ? 2 : min(NH, (int)a.nbn - t.nt * NH);
  };

  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRole));
    if (warp == 0) {
      // ============================ weights (and activations in order)
      Ring st;
      while (!guard.aborted() && walk.take(seg)) {
        const Fp8Tile t = my_tile(seg.tile);
        const int nb = blocks_of(t);
        // a pair's second weight block is the second CTA's; where it lies past N the
        // copy brings zeros, and the pair always runs at the full width
        const uint32_t bytes = CG == 2 ? CG * (kWBytes + (gather ? 0 : kABytes))
                                       : nb * kWBytes + (gather ? 0 : kABytes);
        for (int kb = seg.kb0; kb < seg.kb1; ++kb, st.next(n_stages)) {
          const uint32_t s = st.i;
          bar_wait(&empty[s], st.phase ^ 1, guard);  // the first use passes
          if (guard.aborted()) break;
          if (lane) continue;
          uint8_t *buf = tsm + s * kStage, *dst = buf + kABytes;
          if (rank == 0) bar_expect(&full[s], bytes);
          if (!gather) tma_x<CG>(buf, &maps.x, kb * 128, t.row0, &full[s]);
          if (SWIGLU) {
            if (CG == 2) {
              tma_w<CG>(dst, &maps.w[rank], kb * 128, t.nt * 128, t.e, &full[s]);
            } else {
              tma_w<CG>(dst, &maps.w[0], kb * 128, t.nt * 128, t.e, &full[s]);
              tma_w<CG>(dst + kWBytes, &maps.w[1], kb * 128, t.nt * 128, t.e, &full[s]);
            }
          } else if (CG == 2) {
            tma_w<CG>(dst, &maps.w[0], kb * 128, (t.nt * 2 + rank) * 128, t.e, &full[s]);
          } else {
            for (int h = 0; h < nb; ++h)
              tma_w<CG>(dst + h * kWBytes, &maps.w[0], kb * 128, (t.nt * NH + h) * 128, t.e,
                        &full[s]);
          }
        }
      }
      // the stages still in use: leave with no copy in flight
      for (uint32_t i = 0; i < n_stages; ++i, st.next(n_stages))
        if (!bar_wait_for(*abort_flag && rank == 0 ? &full[st.i] : &empty[st.i], st.phase ^ 1))
          atomicOr(a.err, kErrTimeout);
    } else if (warp == 1 && rank == 0) {
      // ============================ MMA issuer
      Ring st, acc;
      while (!guard.aborted() && walk.take(seg)) {
        const Fp8Tile t = my_tile(seg.tile);
        const uint32_t idesc = idesc_for<CG>(CG == 2 ? 256 : 128 * blocks_of(t));
        for (int kb = seg.kb0; kb < seg.kb1; ++kb, st.next(n_stages), acc.next(2)) {
          const uint32_t s = st.i, b = acc.i;
          bar_wait(&full[s], st.phase, guard);
          bar_wait(&d_empty[b], acc.phase ^ 1, guard);
          // what cp.async wrote is read by the tensor core's proxy
          if (gather) fence_async();
          tc_fence_after();
          const uint64_t ad = sw128_desc(s32(tsm + s * kStage));
          const uint64_t bd = sw128_desc(s32(tsm + s * kStage + kABytes));
          tc_mma_block<CG>(tmem + b * 256, ad, bd, idesc);
          tc_commit<CG>(&empty[s]);
          tc_commit<CG>(&d_full[b]);
        }
      }
      if (guard.aborted()) {  // else the epilogue has waited for every MMA
        tc_commit<CG>(drain);
        bar_wait_for(drain, 0);
      }
    } else if (warp == 1 && gather) {
      // ============================ second CTA: its activations have landed
      Ring st;
      while (!guard.aborted() && walk.take(seg))
        for (int kb = seg.kb0; kb < seg.kb1; ++kb, st.next(n_stages)) {
          bar_wait(&landed[st.i], st.phase, guard);
          fence_async();
          __syncwarp();
          if (lane == 0) bar_arrive_first(&full[st.i]);
        }
    } else if (warp >= 2 && gather) {
      // ============================ activations through perm: in instruction j of
      // MT / 8, warp w copies rows 8j + 4w .. + 3, eight lanes a row of 128 codes
      constexpr int kJ = MT / 8;
      const int r0 = 4 * (warp - 2) + lane / 8, chunk = lane & 7;
      uint64_t *done = rank == 0 ? full : landed;
      Ring st;
      while (!guard.aborted() && walk.take(seg)) {
        const Fp8Tile t = my_tile(seg.tile);
        int row[kJ];  // a bad one (flagged) reads row 0
#pragma unroll
        for (int j = 0; j < kJ; ++j)
          row[j] = 8 * j + r0 < t.rows ? max(0, fp8_x_row(a, t.row0 + 8 * j + r0)) : -1;
        for (int kb = seg.kb0; kb < seg.kb1; ++kb, st.next(n_stages)) {
          const uint32_t s = st.i;
          bar_wait(&empty[s], st.phase ^ 1, guard);
          const uint32_t k0 = kb * 128 + chunk * 16;
          const uint8_t *src = a.xq + (k0 < a.K ? k0 : 0);
          const int bytes = k0 < a.K ? 16 : 0;
          // 128-byte swizzle: chunk c of row r at c ^ (r % 8)
          const uint32_t dst = s32(tsm + s * kStage) + r0 * 128 + ((chunk ^ r0) << 4);
#pragma unroll
          for (int j = 0; j < kJ; ++j)
            cp16(dst + j * 1024, src + (size_t)(uint32_t)row[j] * a.K, bytes, row[j] >= 0);
          cp_arrive(&done[s]);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    // ============================ epilogue
    const int ew = warp - kEpiWarp0, half = ew >> 2, quarter = warp & 3;
    const int m = quarter * 32 + lane;  // row of this CTA's tile, TMEM lane
    // this warp's columns: 64 of each block (SwiGLU, or one block), or one block
    constexpr bool kSplitBlock = SWIGLU || NH == 1;
    constexpr int kChunks = SWIGLU || NH == 2 ? 4 : 2;  // of 32 columns
    const uint32_t col0 = (uint32_t)(quarter * 32) << 16 | (kSplitBlock ? 64 : 128) * half;
    constexpr uint32_t kCol1 = SWIGLU ? 128 : 64;  // from chunk 0 to chunk 2
    uint32_t g = 0, npair = 0;  // accumulators, and meetings of the pair, so far
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) bar_arrive(&pair[quarter]);
      bar_wait(&pair[quarter], npair++ & 1, guard);
    };
    auto release = [&](uint32_t b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2 && rank == 1) bar_arrive_first(&d_empty[b]);
        else bar_arrive(&d_empty[b]);
      }
    };
    uint32_t n_ex = 0;
    while (!guard.aborted() && walk.take(seg)) {
      const Fp8Tile t = my_tile(seg.tile);
      const bool warp_live = quarter * 32 < t.rows && (kSplitBlock || half < blocks_of(t));
      const bool live = warp_live && m < t.rows;
      float2 acc[16 * kChunks];
#pragma unroll
      for (int i = 0; i < 16 * kChunks; ++i) acc[i] = make_float2(0.0f, 0.0f);
      if (!warp_live) {
        for (int kb = seg.kb0; kb < seg.kb1; ++kb, ++g) {
          bar_wait(&d_full[g & 1], (g / 2) & 1, guard);
          release(g & 1);
        }
      } else {
        const int r = t.row0 + min(m, t.rows - 1);
        const size_t blk = kSplitBlock ? t.nt : 2 * t.nt + half;
        const float *xs = a.xs + (size_t)max(0, fp8_x_row(a, r)) * a.nbk;
        const float *wa = a.wsc[0] + ((size_t)t.e * a.nbn + blk) * a.nbk;
        const float *wb = SWIGLU ? a.wsc[1] + ((size_t)t.e * a.nbn + blk) * a.nbk : wa;
        float sx = xs[seg.kb0], sa = wa[seg.kb0], sb = SWIGLU ? wb[seg.kb0] : 0.0f;
        auto fma32 = [&](float (&v)[32], int c, float s) {
          const float2 s2 = make_float2(s, s);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            acc[16 * c + i] = __ffma2_rn(make_float2(v[2 * i], v[2 * i + 1]), s2, acc[16 * c + i]);
        };
        // Two loads of 32 columns are in flight at a time (a wait covers all of a
        // thread's loads), the next pair issued as registers come free -- across
        // the blocks too, so that a load's latency lies under the FMAs before it.
        float v0[32], v1[32];
        bar_wait(&d_full[g & 1], (g / 2) & 1, guard);
        tc_fence_after();
        tc_ld32(tmem + col0 + (g & 1) * 256, v0);
        tc_ld32(tmem + col0 + (g & 1) * 256 + 32, v1);
        for (int kb = seg.kb0; kb < seg.kb1; ++kb, ++g) {
          const uint32_t base = tmem + col0 + (g & 1) * 256;
          const float s0 = sx * sa, s1 = SWIGLU ? sx * sb : s0;
          const int kn = min(kb + 1, seg.kb1 - 1);
          // the next block's scales, on the way while this one is added
          sx = xs[kn], sa = wa[kn];
          if (SWIGLU) sb = wb[kn];
          tc_wait_ld32(v0);
          tie32(v1);
          if (kChunks == 4) {
            fma32(v0, 0, s0);
            tc_ld32(base + kCol1, v0);
            fma32(v1, 1, s0);
            tc_ld32(base + kCol1 + 32, v1);
            tc_wait_ld32(v0);
            tie32(v1);
          }
          release(g & 1);
          fma32(v0, kChunks - 2, s1);
          const bool more = kb + 1 < seg.kb1;
          const uint32_t next = tmem + col0 + ((g + 1) & 1) * 256;
          if (more) {
            bar_wait(&d_full[(g + 1) & 1], ((g + 1) / 2) & 1, guard);
            tc_fence_after();
            tc_ld32(next, v0);
          }
          fma32(v1, kChunks - 1, s1);
          if (more) tc_ld32(next + 32, v1);
        }
      }
      // ---- a share of a tile: the last of its workers adds up all shares
      if (seg.kb1 - seg.kb0 < (int)a.nbk) {
        if (quarter * 32 >= t.rows) continue;  // both warps of the pair
        const int c0 = walk.first_worker(seg.tile);
        const int n = walk.last_worker(seg.tile) - c0 + 1;
        // part of worker c: its second slot if it starts the tile, its first otherwise
        auto part = [&](int c) {
          return (float4 *)(a.part + (size_t)(2 * (c * CG + rank) + (c == c0)) * a.part_stride) +
                 (size_t)(quarter * 2 + half) * 1024 + lane;
        };
        float4 *mine = part(worker);
#pragma unroll
        for (int i = 0; i < 8 * kChunks; ++i)
          __stcg(mine + 32 * i,
                 make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y));
        __threadfence();
        meet();
        uint32_t *count = a.sync + 4 * (seg.tile * CG + rank) + quarter;
        if (half == 0 && lane == 0) {
          __threadfence();
          const bool last = atomicAdd(count, 1u) == (uint32_t)n - 1;
          if (last) atomicExch(count, 0u);
          last_part[quarter] = last;
        }
        meet();
        if (!last_part[quarter]) continue;
        __threadfence();
#pragma unroll
        for (int i = 0; i < 16 * kChunks; ++i) acc[i] = make_float2(0.0f, 0.0f);
        for (int p = 0; p < n; ++p) {
          const float4 *src = part(c0 + p);
#pragma unroll
          for (int i = 0; i < 8 * kChunks; ++i) {
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
        const uint32_t n0 = (uint32_t)t.nt * (128 * NH) + (NH == 2 ? 128 : 64) * half;
        if (vec) {
          if (a.odt == MOE_DT_F32) {
            float *dst = (float *)a.out + (size_t)r * a.ld + n0;
#pragma unroll
            for (int i = 0; i < 4 * kChunks; ++i)
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
            for (int i = 0; i < 2 * kChunks; ++i)
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
          for (int i = 0; i < 16 * kChunks; ++i) {
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
          acc[i].x = fp8_swiglu_value(acc[i].x, acc[(kChunks * 8 + i) % (16 * kChunks)].x);
          acc[i].y = fp8_swiglu_value(acc[i].y, acc[(kChunks * 8 + i) % (16 * kChunks)].y);
          amax = fmaxf(amax, fmaxf(fabsf(acc[i].x), fabsf(acc[i].y)));
        }
        float *e = ex + (n_ex++ & 1) * 256;
        e[128 * half + m] = amax;
        meet();
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
  if (CG == 2) cluster_sync_all();  // no arrival of the other CTA's is still to come
  if (warp == 1) {
    tc_fence_after();
    if (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ---------------------------------------------------------------- host
template <bool SWIGLU, int MT, int NH, int CG>
cudaError_t run_tc(Fp8Args &a, cudaStream_t stream) {
  const int sms = fp8_ctas() / CG * CG;
  fp8_set_tiles(a, SWIGLU ? a.nbn : (a.nbn + NH - 1) / NH, sms / CG);
  const uint32_t quarters = ((a.R < 128 ? a.R : 128) + 31) / 32;
  a.part_stride = (size_t)quarters * 8192;
  Fp8Maps maps;
  memset(&maps, 0, sizeof maps);
  if (!byte_map(&maps.x, a.xq, a.K, a.n_x, 1, 2, MT) ||
      !byte_map(&maps.w[0], a.wq[0], a.K, a.N, a.E, 3, 128) ||
      (SWIGLU && !byte_map(&maps.w[1], a.wq[1], a.K, a.N, a.E, 3, 128)))
    return cudaErrorInvalidValue;
  if (!SWIGLU) maps.w[1] = maps.w[0];
  // 32-byte stores: whole groups of 32 bytes inside every row
  const uint32_t group = 32 / (SWIGLU ? 1 : (uint32_t)dtype_size(a.odt));
  const bool vec = ((uintptr_t)a.out & 31) == 0 && a.N % group == 0 && a.ld % group == 0;
  auto kern = k_fp8_tc<SWIGLU, MT, NH, CG>;
  const size_t stage = MT * 128 + NH / CG * (size_t)kWBytes;
  const size_t rest = 1024 + 512 + 2048 + fp8_tiles_smem(a.E);
  int ns = (int)((kSmemLimit - rest) / stage);
  if (ns > kMaxStages) ns = kMaxStages;
  const size_t smem = rest + ns * stage;
  const int workers = sms / CG;
  const int split_below = workers * 7 / 8;
  static int set[kMaxDevices];
  const cudaError_t e = allow_smem(kern, smem, set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = sms;
  cfg.blockDim = kTcThreads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a, maps, (uint32_t)ns, split_below, vec);
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
  const uint64_t R = a.R, E = a.E;
  if (R <= 192 * E)
    return swiglu ? run_tc<true, 128, 2, 1>(a, stream) : run_tc<false, 128, 2, 1>(a, stream);
  return swiglu ? run_tc<true, 128, 2, 2>(a, stream) : run_tc<false, 128, 2, 2>(a, stream);
}

}  // namespace moe
