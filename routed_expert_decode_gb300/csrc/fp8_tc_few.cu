// fp8_tc_few.cu -- routed products over block-scaled e4m3 operands on the tensor
// cores, for experts with few rows: bound by the stream of weights from HBM.
//
// A tile is NB = 1 or 2 blocks of 128 weight rows (the gate and up rows of one block of
// 128 features, or one or two blocks of the product) by up to MT activation rows of
// one expert.  The weights sit on the MMA's M side and the activation rows on its N side
// (N = MT), so that what the epilogue reads back per block of 128 along K is 128 NB x MT
// sums and not 128 x 128 NB whatever the rows: with the rows on the M side, one row's
// epilogue took ~750 clocks a block against the ~1400 that HBM gives an SM, and each
// wait of the chain showed.  An accumulator takes NB MT of the 512 TMEM columns, and
// 256 / MT of them are in flight.
//
// What it reaches (us, TB/s of weights; a copy reaches 6.79; the GPUs measured differ by 3
// %): one token of 8 experts, d 6144, f 2048: gate/up 34.2-35.5, 5.7-5.9, down 21.5-22.2,
// 4.5-4.7; 512 tokens of 256 experts, gate/up 918-950, 6.8-7.0.  A call's launch and
// prologue are ~5 us of each.
//
// Epilogue warp (q, c) owns features 32q.. of both blocks for rows [c MT/2,
// (c+1) MT/2): per block of K it adds MT/2 columns of each, times scale_w (one
// scalar a weight block) times scale_x (one a row, from shared memory), to fp32 sums
// in registers.  After SwiGLU a row's quantisation block spans the four quarters:
// a warp maximum, and one word a quarter and row in shared memory.
//
// Warps: 0 weights (and rows in order) by TMA, 1 TMEM owner and MMA issuer, 2 routed
// rows by cp.async through perm, 3 the rows' scales, 4..11 epilogue.  The work
// goes out over one CTA per SM as Walk says; the shares of a split tile meet in the
// workspace, where the last to arrive adds all of them in ascending K.
#include <string.h>

#include "fp8_tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kFewThreads = 12 * 32;

template <int N>
struct Int {
  static constexpr int n = N;
};

// N consecutive fp32 columns of this warp's 32 TMEM lanes
template <int N>
struct Cols {
  float v[N];
  __device__ __forceinline__ void load(uint32_t taddr) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    if (N == 32) {
      tc_ld32(taddr, *reinterpret_cast<float (*)[32]>(v));
    } else if (N == 16) {
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
          "%13,%14,%15}, [%16];"
          : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
            "=r"(r[7]), "=r"(r[8 % N]), "=r"(r[9 % N]), "=r"(r[10 % N]), "=r"(r[11 % N]),
            "=r"(r[12 % N]), "=r"(r[13 % N]), "=r"(r[14 % N]), "=r"(r[15 % N])
          : "r"(taddr));
    } else {
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
          : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
            "=r"(r[7])
          : "r"(taddr));
    }
  }
  // no use of the values moves above this point
  __device__ __forceinline__ void tie() {
#pragma unroll
    for (int i = 0; i < N; i += 8)
      asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]),
                   "+f"(v[i + 5]), "+f"(v[i + 6]), "+f"(v[i + 7]));
  }
};

template <bool SWIGLU, int MT, int NB>
__global__ void __launch_bounds__(kFewThreads, 1)
    k_fp8_few(const Fp8Args a, const __grid_constant__ Fp8Maps maps, const uint32_t n_stages,
              const int split_below) {
  pdl_trigger();
  extern __shared__ __align__(1024) uint8_t tsm_raw[];
  uint8_t *tsm = tsm_raw + ((0u - s32(tsm_raw)) & 1023u);  // stays a shared address
  static_assert(!SWIGLU || NB == 2, "gate and up");
  constexpr uint32_t kXBytes = MT * 128, kStage = kXBytes + NB * kWBytes;
  constexpr uint32_t kAccs = 256 / MT;        // accumulators in flight
  constexpr int kC = MT / 2;                  // rows of an epilogue warp
  const int tid = threadIdx.x, lane = tid & 31;
  // through a shuffle, so that the roles' branches are known to be uniform
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  uint8_t *ctrl = tsm + n_stages * kStage;
  uint64_t *full = (uint64_t *)ctrl;    // [kMaxStages] operands of a stage landed
  uint64_t *empty = full + kMaxStages;  // [kMaxStages] ... consumed
  uint64_t *d_full = empty + kMaxStages;  // [kAccs] accumulator and its row scales written
  uint64_t *d_empty = d_full + kAccs;   // [kAccs] ... read
  uint64_t *meet_bar = d_empty + kAccs;  // [2] the four epilogue warps of a row half
  uint64_t *drain = meet_bar + 2;       // the MMAs of an aborted call
  uint32_t *tmem_holder = (uint32_t *)(drain + 1);
  volatile int *abort_flag = (volatile int *)(tmem_holder + 1);
  volatile int *last_part = (volatile int *)(tmem_holder + 2);  // [2]
  float *xsc = (float *)(ctrl + 512);                           // [kAccs][MT] row scales
  float *red = xsc + kAccs * MT;                                // [2][4][MT] row maxima
  int *tiles_sm = (int *)(red + 8 * MT);
  const bool gather = a.perm != nullptr;

  if (tid == 32) {
    prefetch_map(&maps.w[0]);
    prefetch_map(&maps.w[1]);
    if (!gather) prefetch_map(&maps.x);
  }
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      bar_init(&full[i], gather ? 33 : 1);  // the TMA producer, and warp 2's lanes
      bar_init(&empty[i], 1);
    }
    for (uint32_t i = 0; i < kAccs; ++i) {
      bar_init(&d_full[i], 2);   // the MMAs, and the row scales
      bar_init(&d_empty[i], 8);
    }
    for (int i = 0; i < 2; ++i) bar_init(&meet_bar[i], 4);
    bar_init(drain, 1);
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
  fp8_warm(a);
  pdl_wait();
  const RowTiles rt = fp8_row_tiles<MT>(a, tiles_sm);
  Walk walk(rt.total * (int)a.n_tiles, a, (int)blockIdx.x, (int)gridDim.x, split_below);
  Seg seg;
  const Guard guard{a.err, abort_flag};
  // weight blocks that a tile has: the last of an odd number stands alone
  auto blocks_of = [&](const Fp8Tile &t) { return SWIGLU ? 2 : min(NB, (int)a.nbn - t.nt * NB); };

  if (warp == 0) {
    // ============================ weights (and activations in order)
    Ring st;
    while (!guard.aborted() && walk.take(seg)) {
      const Fp8Tile t = fp8_tile<MT>(a, rt, seg.tile);
      const int nb = blocks_of(t);
      const uint32_t bytes = nb * kWBytes + (gather ? 0 : kXBytes);
      for (int kb = seg.kb0; kb < seg.kb1; ++kb, st.next(n_stages)) {
        const uint32_t s = st.i;
        bar_wait(&empty[s], st.phase ^ 1, guard);  // the first use passes
        __syncwarp();
        if (guard.aborted()) break;
        if (lane) continue;
        uint8_t *buf = tsm + s * kStage, *dst = buf + kXBytes;
        bar_expect(&full[s], bytes);
        for (int h = 0; h < nb; ++h)
          tma_w(dst + h * kWBytes, &maps.w[SWIGLU ? h : 0], kb * 128,
                   (SWIGLU ? t.nt : t.nt * NB + h) * 128, t.e, &full[s]);
        if (!gather) tma_x(buf, &maps.x, kb * 128, t.row0, &full[s]);
      }
    }
    // the stages still in use: leave with no copy in flight
    for (uint32_t i = 0; i < n_stages; ++i, st.next(n_stages))
      if (!bar_wait_for(*abort_flag ? &full[st.i] : &empty[st.i], st.phase ^ 1))
        atomicOr(a.err, kErrTimeout);
  } else if (warp == 1) {
    // ============================ MMA issuer
    Ring st, acc;
    const uint32_t idesc = idesc_for(MT);
    while (!guard.aborted() && walk.take(seg)) {
      const int nb = blocks_of(fp8_tile<MT>(a, rt, seg.tile));
      for (int kb = seg.kb0; kb < seg.kb1; ++kb, st.next(n_stages), acc.next(kAccs)) {
        bar_wait(&full[st.i], st.phase, guard);
        bar_wait(&d_empty[acc.i], acc.phase ^ 1, guard);
        if (gather) fence_async();  // cp.async's writes, read by the tensor core's proxy
        tc_fence_after();
        __syncwarp();
        const uint32_t buf = s32(tsm + st.i * kStage);
        const uint64_t xd = sw128_desc(buf), wd = sw128_desc(buf + kXBytes);
        const uint32_t d = tmem + acc.i * NB * MT;
        tc_mma_block(d, wd, xd, idesc);
        if (NB == 2 && nb == 2) tc_mma_block(d + MT, wd + (kWBytes >> 4), xd, idesc);
        tc_commit(&empty[st.i]);
        tc_commit(&d_full[acc.i]);
      }
    }
    if (guard.aborted()) {  // else the epilogue has waited for every MMA
      tc_commit(drain);
      bar_wait_for(drain, 0);
    }
  } else if (warp == 2) {
    if (gather) {
      // ============================ activations through perm: in instruction j of MT
      // / 4, rows 4j .. + 3, eight lanes a row of 128 codes
      constexpr int kJ = MT / 4;
      const int r0 = lane / 8, chunk = lane & 7;
      Ring st;
      while (!guard.aborted() && walk.take(seg)) {
        const Fp8Tile t = fp8_tile<MT>(a, rt, seg.tile);
        int row[kJ];  // a bad one (flagged) reads row 0
#pragma unroll
        for (int j = 0; j < kJ; ++j)
          row[j] = 4 * j + r0 < t.rows ? max(0, fp8_x_row(a, t.row0 + 4 * j + r0)) : -1;
        for (int kb = seg.kb0; kb < seg.kb1; ++kb, st.next(n_stages)) {
          bar_wait(&empty[st.i], st.phase ^ 1, guard);
          const uint32_t k0 = kb * 128 + chunk * 16;
          const uint8_t *src = a.xq + (k0 < a.K ? k0 : 0);
          const int bytes = k0 < a.K ? 16 : 0;
          const uint32_t buf = s32(tsm + st.i * kStage);
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            // 128-byte swizzle: chunk c of row r at c ^ (r % 8)
            const int r = 4 * j + r0;
            cp16(buf + r * 128 + ((chunk ^ (r & 7)) << 4), src + (size_t)(uint32_t)row[j] * a.K,
                 bytes, row[j] >= 0);
          }
          cp_arrive(&full[st.i]);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else if (warp == 3) {
    // ============================ row scales, one block of K ahead in registers
    constexpr int kR = MT / 32;
    Ring acc;
    while (!guard.aborted() && walk.take(seg)) {
      const Fp8Tile t = fp8_tile<MT>(a, rt, seg.tile);
      const float *xs[kR];
      float next[kR];
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const int r = min(lane + 32 * i, t.rows - 1);
        xs[i] = a.xs + (size_t)max(0, fp8_x_row(a, t.row0 + r)) * a.nbk;
        next[i] = xs[i][seg.kb0];
      }
      for (int kb = seg.kb0; kb < seg.kb1; ++kb, acc.next(kAccs)) {
        float v[kR];
#pragma unroll
        for (int i = 0; i < kR; ++i) {
          v[i] = next[i];
          next[i] = xs[i][min(kb + 1, seg.kb1 - 1)];
        }
        bar_wait(&d_empty[acc.i], acc.phase ^ 1, guard);
#pragma unroll
        for (int i = 0; i < kR; ++i) xsc[acc.i * MT + lane + 32 * i] = v[i];
        __syncwarp();
        if (lane == 0) bar_arrive(&d_full[acc.i]);
      }
    }
  } else {
    // ============================ epilogue
    const int ew = warp - 4, c = ew >> 2, quarter = warp & 3;
    const int f = quarter * 32 + lane;  // feature of a weight block, TMEM lane
    Ring dr;
    uint32_t nmeet = 0, nred = 0;
    auto meet = [&]() {  // the four warps of this row half
      __syncwarp();
      if (lane == 0) bar_arrive(&meet_bar[c]);
      bar_wait(&meet_bar[c], nmeet++ & 1, guard);
    };
    const uint32_t col0 = ((uint32_t)(quarter * 32) << 16) + c * kC;
    while (!guard.aborted() && walk.take(seg)) {
      const Fp8Tile t = fp8_tile<MT>(a, rt, seg.tile);
      const int rows = t.rows - c * kC;  // live rows of this warp
      const int nb = blocks_of(t);
      float2 acc[NB][kC / 2];  // pairs of rows
#pragma unroll
      for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int i = 0; i < kC / 2; ++i) acc[h][i] = make_float2(0.0f, 0.0f);
      // the segment's blocks of K with NC columns read of each accumulator
      auto add = [&](auto nc) {
        constexpr int NC = decltype(nc)::n;
        const size_t blk = SWIGLU ? t.nt : NB * t.nt;
        const float *wa = a.wsc[0] + ((size_t)t.e * a.nbn + blk) * a.nbk;
        const float *wb = SWIGLU ? a.wsc[1] + ((size_t)t.e * a.nbn + blk) * a.nbk
                          : nb == 2 ? wa + a.nbk : wa;
        float sa = wa[seg.kb0], sb = wb[seg.kb0];
        for (int kb = seg.kb0; kb < seg.kb1; ++kb) {
          const float s[2] = {sa, sb};
          const int kn = min(kb + 1, seg.kb1 - 1);
          sa = wa[kn];  // on the way while this block is added
          bar_wait(&d_full[dr.i], dr.phase, guard);
          tc_fence_after();
          __syncwarp();  // each lane waits for itself, the loads take the whole warp
          if (NB == 2) sb = wb[kn];
          Cols<NC> v[NB];
          const uint32_t base = tmem + col0 + dr.i * NB * MT;
          v[0].load(base);
          if (NB == 2) v[NB - 1].load(base + MT);
          float4 x[NC / 4];
          const float4 *xp = (const float4 *)(xsc + dr.i * MT + c * kC);
#pragma unroll
          for (int i = 0; i < NC / 4; ++i) x[i] = xp[i];
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          v[0].tie();
          if (NB == 2) v[NB - 1].tie();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&d_empty[dr.i]);
          dr.next(kAccs);
#pragma unroll
          for (int h = 0; h < NB; ++h) {
            const float2 s2 = make_float2(s[h], s[h]);
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) {
              const float4 q = x[i / 2];
              const float2 xx = i & 1 ? make_float2(q.z, q.w) : make_float2(q.x, q.y);
              acc[h][i] = __ffma2_rn(make_float2(v[h].v[2 * i], v[h].v[2 * i + 1]),
                                     __fmul2_rn(xx, s2), acc[h][i]);
            }
          }
        }
      };
      if (rows <= 0) {
        for (int kb = seg.kb0; kb < seg.kb1; ++kb, dr.next(kAccs)) {
          bar_wait(&d_full[dr.i], dr.phase, guard);
          __syncwarp();
          if (lane == 0) bar_arrive(&d_empty[dr.i]);
        }
      } else if (rows <= 8) {
        add(Int<8>());
      } else {
        add(Int<kC>());
      }
      if (rows <= 0) continue;  // the four warps of this half alike
      // ---- a share of a tile: the last of its workers adds up all shares
      if (seg.kb1 - seg.kb0 < (int)a.nbk) {
        const int c0 = walk.first_worker(seg.tile);
        const int n = walk.last_worker(seg.tile) - c0 + 1;
        // part of worker c: its second slot if it starts the tile, its first otherwise
        auto part = [&](int w) {
          return (float2 *)(a.part + (size_t)(2 * w + (w == c0)) * a.part_stride) +
                 (size_t)ew * (kC * 32) + lane;
        };
        float2 *mine = part((int)blockIdx.x);
#pragma unroll
        for (int h = 0; h < NB; ++h)
#pragma unroll
          for (int i = 0; i < kC / 2; ++i)
            if (2 * i < rows) __stcg(mine + (h * (kC / 2) + i) * 32, acc[h][i]);
        __threadfence();
        meet();
        uint32_t *count = a.sync + 4 * seg.tile + c;
        if (quarter == 0 && lane == 0) {
          __threadfence();
          const bool last = atomicAdd(count, 1u) == (uint32_t)n - 1;
          if (last) atomicExch(count, 0u);
          last_part[c] = last;
        }
        meet();
        if (!last_part[c]) continue;
        __threadfence();
#pragma unroll
        for (int h = 0; h < NB; ++h)
#pragma unroll
          for (int i = 0; i < kC / 2; ++i) acc[h][i] = make_float2(0.0f, 0.0f);
#pragma unroll 4
        for (int p = 0; p < n; ++p) {  // four shares' loads on the way together
          const float2 *src = part(c0 + p);
#pragma unroll
          for (int h = 0; h < NB; ++h)
#pragma unroll
            for (int i = 0; i < kC / 2; ++i)
              if (2 * i < rows) {
                const float2 v = __ldcg(src + (h * (kC / 2) + i) * 32);
                acc[h][i].x += v.x;
                acc[h][i].y += v.y;
              }
        }
      }
      // ---- outputs: a warp's lanes are consecutive columns of a row
      const int r0 = t.row0 + c * kC;
      if (!SWIGLU) {
#pragma unroll
        for (int h = 0; h < NB; ++h) {
          const uint32_t n = (uint32_t)(t.nt * NB + h) * 128 + f;
          if (n >= a.N) continue;
          const size_t at = (size_t)r0 * a.ld + n;
          auto store = [&](auto *p, auto from) {
            p += at;
#pragma unroll
            for (int i = 0; i < kC; ++i) {
              if (i >= rows) break;
              p[(size_t)i * a.ld] = from(i & 1 ? acc[h][i / 2].y : acc[h][i / 2].x);
            }
          };
          if (a.odt == MOE_DT_F32) store((float *)a.out, [](float v) { return v; });
          else if (a.odt == MOE_DT_BF16) store((__nv_bfloat16 *)a.out, Elem<MOE_DT_BF16>::from);
          else store((__half *)a.out, Elem<MOE_DT_F16>::from);
        }
      } else {
        // h (past N: g = u = 0), its maxima over this warp's 32 features, then over
        // the quarters'; |h| of numbers orders as its bit pattern
        float *mx = red + (nred++ & 1) * 4 * MT + c * kC;
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          if (i >= rows) break;  // past the code of the rows that are not there
          float &g = i & 1 ? acc[0][i / 2].y : acc[0][i / 2].x;
          g = fp8_swiglu_value(g, i & 1 ? acc[NB - 1][i / 2].y : acc[NB - 1][i / 2].x);
          const float m = g == g ? fabsf(g) : 0.0f;
          const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
          if (lane == 0) mx[quarter * MT + i] = __uint_as_float(w);
        }
        meet();
        // lane i works out row i's scale
        float sc = 0.0f, inv = 0.0f;
        if (lane < rows && lane < kC) {
          const float *q = mx + lane;
          fp8_block_scale(fmaxf(fmaxf(q[0], q[MT]), fmaxf(q[2 * MT], q[3 * MT])), sc, inv);
          if (quarter == 0) a.hs[(size_t)(r0 + lane) * a.nbn + t.nt] = sc;
        }
        const uint32_t n = (uint32_t)t.nt * 128 + f;
        uint8_t *dst = (uint8_t *)a.out + (size_t)r0 * a.N + n;
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          if (i >= rows) break;
          const float g = i & 1 ? acc[0][i / 2].y : acc[0][i / 2].x;
          const uint8_t q = e4m3x1(g * __shfl_sync(0xffffffffu, inv, i));
          if (n < a.N) dst[(size_t)i * a.N] = q;
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

template <bool SWIGLU, int MT, int NB>
cudaError_t run_few(Fp8Args &a, cudaStream_t stream) {
  const int sms = fp8_ctas();
  fp8_set_tiles(a, SWIGLU ? a.nbn : (a.nbn + NB - 1) / NB, sms);
  a.part_stride = (size_t)MT * 256;
  if (a.part_stride * 4 > fp8_part_bytes(a.R)) return cudaErrorInvalidValue;
  Fp8Maps maps;
  memset(&maps, 0, sizeof maps);
  if (!byte_map(&maps.x, a.xq, a.K, a.n_x, 1, 2, MT) ||
      !byte_map(&maps.w[0], a.wq[0], a.K, a.N, a.E, 3, 128) ||
      (SWIGLU && !byte_map(&maps.w[1], a.wq[1], a.K, a.N, a.E, 3, 128)))
    return cudaErrorInvalidValue;
  if (!SWIGLU) maps.w[1] = maps.w[0];
  auto kern = k_fp8_few<SWIGLU, MT, NB>;
  const size_t stage = MT * 128 + NB * (size_t)kWBytes;
  const size_t rest = 1024 + 512 + 4 * (256 + 8 * MT) + fp8_tiles_smem(a.E);
  int ns = (int)((kSmemLimit - rest) / stage);
  if (ns > kMaxStages) ns = kMaxStages;
  const size_t smem = rest + ns * stage;
  static std::atomic<bool> done[kMaxDevices];
  const cudaError_t e = allow_smem(kern, done);
  if (e != cudaSuccess) return e;
  // Tiles are split along K when they leave three SMs of four idle and K has 16 blocks:
  // 64 SMs already draw 5.4 TB/s, and under a saturated HBM each of the split's round
  // trips (shares out, count, shares in) takes ~3 us.  Tiles of 128 columns, split and
  // whole: K 6144, 4 tiles 7.4 and 13.5 us, 32 tiles 10.6 and 13.8, 64 tiles 16.9 and 14.7;
  // K 2048, 4 tiles 5.9 and 6.3; K 1024, 4 tiles 5.6 and 4.8.  Between 32 and 64, through
  // the binding: 40 tiles of K 6144 12.3 and 15.0, of K 2048 9.2 and 7.6, and 40 tiles of 256
  // columns after a round of whole ones (one token's down product, K 2048) 26.6 and 22.0.
  return launch_k(kern, sms, kFewThreads, smem, stream, true, a, maps, (uint32_t)ns,
                  a.nbk >= 16 ? sms / 4 : 0);
}

}  // namespace

cudaError_t launch_fp8_few(Fp8Args &a, bool swiglu, cudaStream_t stream) {
  const uint64_t R = a.R, E = a.E;
  if (swiglu) return run_few<true, 32, 2>(a, stream);
  if (R > kFp8FewProduct32 * E) return run_few<false, 64, 2>(a, stream);
  // At most this many pairs of weight blocks have rows.  Where every block finds an SM,
  // one a tile draws from more of them (K 2048, 48 pairs: 7.2 against 8.0 us); beyond, a
  // pair shares a tile's fixed work (96 pairs: 13.6 against 11.9 us).
  const uint64_t pairs = (R < E ? R : E) * ((a.nbn + 1) / 2);
  return 2 * pairs <= (uint64_t)fp8_ctas() ? run_few<false, 32, 1>(a, stream)
                                           : run_few<false, 32, 2>(a, stream);
}

}  // namespace moe
