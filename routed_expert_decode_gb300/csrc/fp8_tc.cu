// fp8_tc.cu -- routed and dense products over block-scaled e4m3 operands on the
// 5th-generation tensor cores, for experts with many rows: bound by L2 and arithmetic.
//
// A tile is 128 activation rows of one expert by two blocks of 128 weight rows (256
// columns of the product, or the gate and up rows of one block of 128 features).
// Per block of 128 along K, tcgen05.mma kind::f8f6f4 (M = 128, N = 256, K = 32 four
// times) forms the unscaled products in one of two TMEM accumulators, and the
// epilogue warps add them, times scale_x * scale_w, to fp32 sums in registers: the
// scales change every 128 K, so each accumulator is read once per block.  The
// activation rows sit on the MMA's M side, so that an epilogue thread owns one row:
// its scale product is one scalar per block and matrix, a pair of columns costs one
// packed FMA, and a row's quantisation block after SwiGLU is a maximum over two
// threads' registers.
//
// What bounds it: the operands' way into the SM.  16384 rows of gate/up (d 6144, f 2048,
// 16 experts) take 339 us after a pause, 2.43 PFLOP/s, and 310 with an epilogue that only
// releases the accumulators; 4000 x 4096 x 6144 dense 82 us, 2.45 PFLOP/s, and 77.  48 KB a
// block in 900 to 950 clocks is 52 to 55 of the 64 bytes a clock that L2 gives an SM.  (In
// a steady stream of calls the card's power cap makes them 375-392 us, 2.1-2.2 PFLOP/s,
// and 86-89, 2.3.)  The chain MMA -> loads -> FMAs -> release -> MMA with two
// accumulators to hide it in comes next, so the latency of single instructions counts:
// the buffers are addressed as shared memory and the roles branch on a uniform warp
// number (through generic addresses 430 us and 115, on tid / 32 377 and 107).
// Measured and not kept: pairs of CTAs on 256 rows (cta_group::2, which halves an SM's
// weight bytes: 504 and 122 against 476 and 119 us -- the other CTA's arrivals lengthen
// the chain); accumulators of one weight block each, four in flight (494 and 131:
// the MMA's issue and waits double); TMA's gather of four rows for the routed
// activations (78 clocks a request, 2500 a tile of 128 rows and block).
//
// Routed activation rows are copied by 16-byte cp.async through perm into the
// swizzled layout, so no permuted copy of the activations is written; rows in
// order come by one TMA box.  The scales follow by 4-byte cp.async: loads of them in
// the epilogue took 9 % of the kernel however far ahead they were issued.
//
// Warps: 0 weights and scales, 1 TMEM owner and MMA issuer, 2 and 3 routed activations,
// 4..11 epilogue (warp w reads TMEM lanes 32*(w%4).., columns by half).
//
// Work goes out over one CTA per SM: whole tiles in rounds, and the tiles of the last,
// partial round in two shares along K if every share finds a CTA and K is long.  The
// shares of a tile meet in the workspace: each CTA writes its fp32 sums, the second to
// arrive adds the other's; a sum of two does not depend on their order.  A meeting takes
// ~6.5 us, mostly for 128 KB out of an SM and into another.  Columns 4096, K 6144, 16, 160
// and 512 tiles: 19.9, 42.4 and 85.3 us split, 22.3, 44.5 and 87.0 whole; K 2048, 16
// tiles: 13.3 split, 10.6 whole; four shares of K 6144: 22.0, 43.5 and 85.6.
#include <string.h>

#include "fp8_tc_ptx.cuh"

namespace moe {
namespace {

// a product that stays where it is written: after the loads of its factors have had time
__device__ __forceinline__ float mul_here(float a, float b) {
  float r;
  asm volatile("mul.rn.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

constexpr int kTcThreads = 12 * 32;
constexpr uint32_t kTcStages = 4;  // of the operand ring, at most
constexpr int kEpiWarp0 = 4;
constexpr int kM = 128;  // rows of a tile
// Blocks of K from which the tiles of the last round are split.  Dense, split and whole (us):
//   blocks             32           36           40           48
//   16 tiles       15.7  15.8   16.4  17.1   16.9  18.5   18.3  21.2
//   76             20.0  17.2   21.0  19.1   21.3  21.0   22.8  24.4
//   152 and 16     32.0  31.4   34.3  34.2   35.4  37.2   39.9  43.0
constexpr int kSplitBlocks = 40;
// Scales of the blocks of K in flight.  A block's are written when the MMA a ring of
// stages earlier is done, which was issued when the epilogue had read the block two
// before that: the slot of the block two further back is free.
constexpr uint32_t kScaleSlots = 8;
static_assert(kTcStages + 3 <= kScaleSlots, "a slot's last reader is done");
constexpr uint32_t kABytes = kM * 128, kStage = kABytes + 2 * kWBytes;
// registers per thread after the split: 128 * 72 + 256 * 216 = 384 * 168, the launch's;
// with 56 the activations' row numbers spill (437 against 429 us)
constexpr int kRegsRole = 72, kRegsEpi = 216;

// A CTA's work: half of a split tile, then whole tiles.
struct TileWalk {
  int n_all, kbs, grid, worker, next;
  bool half;  // half a tile is to come
  __device__ TileWalk(int n_all_, const Fp8Args &a, int worker_, int grid_)
      : n_all(n_all_), kbs((int)a.nbk), grid(grid_), worker(worker_) {
    const int rest = n_all - grid * (int)quotient(n_all, grid, a.workers_inv);
    const bool split = 2 * rest <= grid && kbs >= kSplitBlocks;
    half = split && worker < 2 * rest;
    next = (split ? rest : 0) + worker;
  }
  __device__ bool take(Seg &s) {
    if (!half && next >= n_all) return false;
    s.tile = half ? worker >> 1 : next;
    s.kb0 = half && (worker & 1) ? kbs >> 1 : 0;
    s.kb1 = half && !(worker & 1) ? kbs >> 1 : kbs;
    if (!half) next += grid;
    half = false;
    return true;
  }
};

// A row's product over one segment leaves 128 fp32 sums in each of its two epilogue
// threads: acc[0..31] and acc[32..63] are pairs of columns -- of the gate and the
// up block (SwiGLU), or of a block's two halves.
template <bool SWIGLU>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_fp8_tc(const Fp8Args a, const __grid_constant__ Fp8Maps maps, const uint32_t n_stages,
             const bool vec) {
  pdl_trigger();
  extern __shared__ __align__(1024) uint8_t tsm_raw[];
  uint8_t *tsm = tsm_raw + ((0u - s32(tsm_raw)) & 1023u);  // stays a shared address
  const int tid = threadIdx.x, lane = tid & 31;
  // through a shuffle, so that the roles' branches are known to be uniform
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  uint8_t *ctrl = tsm + n_stages * kStage;
  uint64_t *full = (uint64_t *)ctrl;     // [kMaxStages] operands of a stage landed
  uint64_t *empty = full + kMaxStages;   // [kMaxStages] ... consumed
  uint64_t *d_full = empty + kMaxStages;  // [2] accumulator written
  uint64_t *d_empty = d_full + 2;        // [2] ... read
  uint64_t *pair = d_empty + 2;          // [4] the two epilogue warps of a lane quarter
  uint64_t *drain = pair + 4;            // the MMAs of an aborted call
  uint32_t *tmem_holder = (uint32_t *)(drain + 1);
  volatile int *abort_flag = (volatile int *)(tmem_holder + 1);
  volatile int *last_part = (volatile int *)(tmem_holder + 2);  // [4]
  float *ex = (float *)(ctrl + 512);                            // [2][2][128] row maxima
  float *xsc = ex + 512;                                        // [slots][128] row scales
  float *wsc = xsc + kScaleSlots * kM;                          // [slots][2] weight scales
  int *tiles_sm = (int *)(wsc + kScaleSlots * 2);
  const bool gather = a.perm != nullptr;

  if (tid == 32) {
    prefetch_map(&maps.w[0]);
    prefetch_map(&maps.w[1]);
    if (!gather) prefetch_map(&maps.x);
  }
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      // the TMA producer, its warp's scales, and warps 2 and 3
      bar_init(&full[i], 1 + 32 + (gather ? 64 : 0));
      bar_init(&empty[i], 2);  // the MMAs' reads, and the MMA warp
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&d_full[i], 2);  // the MMAs' results, and the MMA warp
      bar_init(&d_empty[i], 8);
    }
    for (int i = 0; i < 4; ++i) bar_init(&pair[i], 2);
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
  const RowTiles rt = fp8_row_tiles<kM>(a, tiles_sm);
  const int worker = (int)blockIdx.x;
  TileWalk walk(rt.total * (int)a.n_tiles, a, worker, (int)gridDim.x);
  Seg seg;
  const Guard guard{a.err, abort_flag};
  auto my_tile = [&](int v) { return fp8_tile<kM>(a, rt, v); };
  // weight blocks that a tile has: the last of an odd number stands alone
  auto blocks_of = [&](const Fp8Tile &t) { return SWIGLU ? 2 : min(2, (int)a.nbn - t.nt * 2); };

  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRole));
    if (warp == 0 || (warp == 2 && !gather)) {
      // ============================ weights (and activations in order), by warp 0;
      // the scales by warp 2 where it has no activations to copy
      const bool scales = gather == (warp == 0);
      Ring st;
      uint32_t slot = 0;
      while (!guard.aborted() && walk.take(seg)) {
        const Fp8Tile t = my_tile(seg.tile);
        const int nb = blocks_of(t);
        const uint32_t bytes = nb * kWBytes + (gather ? 0 : kABytes);
        // scales, by 4-byte copies that land with the stage's operands: four rows a
        // lane, and the two weight blocks'
        const float *xs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = min(lane + 32 * i, t.rows - 1);
          xs[i] = a.xs + (size_t)max(0, fp8_x_row(a, t.row0 + r)) * a.nbk;
        }
        const float *ws = a.wsc[SWIGLU ? lane & 1 : 0] +
                          ((size_t)t.e * a.nbn + (SWIGLU ? t.nt : 2 * t.nt + min(lane & 1, nb - 1))) *
                              a.nbk;
        for (int kb = seg.kb0; kb < seg.kb1; ++kb, st.next(n_stages)) {
          const uint32_t s = st.i;
          bar_wait(&empty[s], st.phase ^ 1, guard);  // the first use passes
          if (guard.aborted()) break;
          if (scales) {
#pragma unroll
            for (int i = 0; i < 4; ++i) cp4(s32(xsc + slot * kM + lane + 32 * i), xs[i] + kb);
            if (lane < 2) cp4(s32(wsc + 2 * slot + lane), ws + kb);
            cp_arrive(&full[s]);
            slot = (slot + 1) % kScaleSlots;
          }
          if (lane || warp) continue;
          uint8_t *buf = tsm + s * kStage, *dst = buf + kABytes;
          bar_expect(&full[s], bytes);
          if (!gather) tma_x(buf, &maps.x, kb * 128, t.row0, &full[s]);
          for (int h = 0; h < nb; ++h)
            tma_w(dst + h * kWBytes, &maps.w[SWIGLU ? h : 0], kb * 128,
                  (SWIGLU ? t.nt : t.nt * 2 + h) * 128, t.e, &full[s]);
        }
      }
      // the stages still in use: leave with no copy in flight
      asm volatile("cp.async.wait_all;" ::: "memory");
      for (uint32_t i = 0; warp == 0 && i < n_stages; ++i, st.next(n_stages))
        if (!bar_wait_for(*abort_flag ? &full[st.i] : &empty[st.i], st.phase ^ 1))
          atomicOr(a.err, kErrTimeout);
    } else if (warp == 1) {
      // ============================ MMA issuer
      Ring st, acc;
      while (!guard.aborted() && walk.take(seg)) {
        const uint32_t idesc = idesc_for(128 * blocks_of(my_tile(seg.tile)));
        for (int kb = seg.kb0; kb < seg.kb1; ++kb, st.next(n_stages), acc.next(2)) {
          const uint32_t buf = s32(tsm + st.i * kStage);
          bar_wait(&full[st.i], st.phase, guard);
          // what cp.async wrote is read by the tensor core's proxy
          if (gather) fence_async();
          bar_wait(&d_empty[acc.i], acc.phase ^ 1, guard);
          tc_fence_after();
          __syncwarp();
          tc_mma_block(tmem + acc.i * 256, sw128_desc(buf), sw128_desc(buf + kABytes), idesc);
          tc_commit(&empty[st.i]);
          tc_commit(&d_full[acc.i]);
          // The scales' way through shared memory: their copies (full, waited for
          // above) come before the epilogue's loads of them, and its loads of two
          // blocks ago (d_empty, likewise) before the copies into their slots.
          bar_arrive_elect(&empty[st.i]);
          bar_arrive_elect(&d_full[acc.i]);
        }
      }
      if (guard.aborted()) {  // else the epilogue has waited for every MMA
        tc_commit(drain);
        bar_wait_for(drain, 0);
      }
    } else if (warp >= 2 && gather) {
      // ============================ activations through perm: in instruction j of
      // 16, warp w copies rows 8j + 4w .. + 3, eight lanes a row of 128 codes
      constexpr int kJ = kM / 8;
      const int r0 = 4 * (warp - 2) + lane / 8, chunk = lane & 7;
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
          cp_arrive(&full[s]);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    // ============================ epilogue
    const int ew = warp - kEpiWarp0, half = ew >> 2, quarter = warp & 3;
    const int m = quarter * 32 + lane;  // row of this CTA's tile, TMEM lane
    // this warp's columns, in chunks of 32: 64 of each weight block (SwiGLU, whose
    // gate and up meet in a thread), or one block's 128
    const uint32_t col0 =
        tmem + ((uint32_t)(quarter * 32) << 16) + (SWIGLU ? 64 : 128) * half;
    constexpr uint32_t kCol2 = SWIGLU ? 128 : 64;  // from chunk 0 to chunk 2
    uint32_t npair = 0;  // meetings of the pair so far
    Ring dr;             // accumulators
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) bar_arrive(&pair[quarter]);
      bar_wait(&pair[quarter], npair++ & 1, guard);
    };
    auto release = [&](uint32_t b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&d_empty[b]);
    };
    uint32_t n_ex = 0, slot = 0;
    while (!guard.aborted() && walk.take(seg)) {
      const Fp8Tile t = my_tile(seg.tile);
      const bool warp_live = quarter * 32 < t.rows && (SWIGLU || half < blocks_of(t));
      const bool live = warp_live && m < t.rows;
      float2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.0f, 0.0f);
      if (!warp_live) {
        for (int kb = seg.kb0; kb < seg.kb1; ++kb, dr.next(2)) {
          bar_wait(&d_full[dr.i], dr.phase, guard);
          release(dr.i);
        }
        slot = (slot + seg.kb1 - seg.kb0) % kScaleSlots;
      } else {
        // columns 32c + 2 [i0, i1) of this warp's, scaled, to the sums
        auto fma = [&](const float (&v)[32], int c, int i0, int i1, float s) {
          const float2 s2 = make_float2(s, s);
#pragma unroll
          for (int i = i0; i < i1; ++i)
            acc[16 * c + i] = __ffma2_rn(make_float2(v[2 * i], v[2 * i + 1]), s2, acc[16 * c + i]);
        };
        // One load of 32 columns is in flight while the chunk before it is added (a wait
        // covers all of a thread's loads), across the blocks too.  The next block's
        // barrier is looked at, and its scales loaded, under the last chunk's FMAs
        // (gate/up 357 -> 347 us; a look that may suspend the warp: 370).
        float v0[32], v1[32], sx, w0, w1 = 0.0f;
        auto scales = [&]() {
          sx = xsc[slot * kM + m];
          w0 = wsc[2 * slot + (SWIGLU ? 0 : half)];
          if (SWIGLU) w1 = wsc[2 * slot + 1];
          slot = (slot + 1) % kScaleSlots;
        };
        bar_wait(&d_full[dr.i], dr.phase, guard);
        tc_fence_after();
        __syncwarp();  // each lane waits for itself, the load takes the whole warp
        tc_ld32(col0 + dr.i * 256, v0);
        scales();
        for (int kb = seg.kb0; kb < seg.kb1; ++kb) {
          const uint32_t col = col0 + dr.i * 256;
          const float s0 = mul_here(sx, w0), s1 = SWIGLU ? mul_here(sx, w1) : s0;
          tc_wait_ld32(v0);
          tc_ld32(col + 32, v1);
          fma(v0, 0, 0, 16, s0);
          tc_wait_ld32(v1);
          tc_ld32(col + kCol2, v0);
          fma(v1, 1, 0, 16, s0);
          tc_wait_ld32(v0);
          tc_ld32(col + kCol2 + 32, v1);
          fma(v0, 2, 0, 16, s1);
          tc_wait_ld32(v1);
          release(dr.i);
          dr.next(2);
          const bool ready = bar_test(&d_full[dr.i], dr.phase);
          fma(v1, 3, 0, 8, s1);
          if (kb + 1 < seg.kb1) {
            if (!ready) bar_wait(&d_full[dr.i], dr.phase, guard);
            tc_fence_after();
            __syncwarp();
            tc_ld32(col0 + dr.i * 256, v0);
            scales();
          }
          fma(v1, 3, 8, 16, s1);
        }
      }
      // ---- half a tile: add the other half, or leave the sums to it
      if (seg.kb1 - seg.kb0 < (int)a.nbk) {
        if (quarter * 32 >= t.rows) continue;  // both warps of the pair
        auto part = [&](int w) {
          return (float4 *)(a.part + (size_t)w * a.part_stride) +
                 (size_t)(quarter * 2 + half) * 1024 + lane;
        };
        float4 *to = part(worker);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          __stcg(to + 32 * i,
                 make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y));
        __threadfence();
        meet();
        if (half == 0 && lane == 0) {
          uint32_t *count = a.sync + 4 * seg.tile + quarter;
          __threadfence();
          const bool second = atomicAdd(count, 1u) == 1u;
          if (second) atomicExch(count, 0u);
          last_part[quarter] = second;
        }
        meet();
        if (!last_part[quarter]) continue;
        __threadfence();
        const float4 *from = part(worker ^ 1);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float4 v = __ldcg(from + 32 * i);
          acc[2 * i].x += v.x;
          acc[2 * i].y += v.y;
          acc[2 * i + 1].x += v.z;
          acc[2 * i + 1].y += v.w;
        }
      }
      // ---- outputs
      const int r = t.row0 + m;
      if (!SWIGLU) {
        if (!warp_live) continue;
        const uint32_t n0 = (uint32_t)(t.nt * 2 + half) * 128;
        // Chunks of 32 bytes of a row.  Two lanes exchange one of each two of theirs, so
        // that a store covers 64 bytes of 16 rows and not 32 of 32 (4000 x 4096 dense: 84.4
        // -> 82.3 us; four lanes and 128 bytes: the same).
        auto store = [&](auto *out, auto pack) {
          constexpr int kC = 32 / sizeof(*out);  // columns of a chunk
          const int odd = lane & 1, pm = m - odd;
#pragma unroll
          for (int i = 0; i < 128 / kC; i += 2) {
            uint32_t w[2][8];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int j = 0; j < 8; ++j) w[h][j] = pack((i + h) * 8 + j);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w[0][j] : w[1][j], 1);
              w[0][j] = odd ? got : w[0][j];
              w[1][j] = odd ? w[1][j] : got;
            }
            const uint32_t n = n0 + kC * (i + odd);
            auto *dst = out + (size_t)(t.row0 + pm) * a.ld + n;
            if (n < a.N && pm < t.rows) st_global32(dst, w[0]);
            if (n < a.N && pm + 1 < t.rows) st_global32(dst + a.ld, w[1]);
          }
        };
        if (vec && a.odt == MOE_DT_F32) {
          store((float *)a.out,
                [&](int i) { return __float_as_uint(i & 1 ? acc[i / 2].y : acc[i / 2].x); });
        } else if (vec && a.odt == MOE_DT_BF16) {
          store((uint16_t *)a.out, [&](int i) { return pack2<MOE_DT_BF16>(acc[i].x, acc[i].y); });
        } else if (vec) {
          store((uint16_t *)a.out, [&](int i) { return pack2<MOE_DT_F16>(acc[i].x, acc[i].y); });
        } else if (live) {
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
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ---------------------------------------------------------------- host
template <bool SWIGLU>
cudaError_t run_tc(Fp8Args &a, cudaStream_t stream) {
  const int sms = fp8_ctas();
  fp8_set_tiles(a, SWIGLU ? a.nbn : (a.nbn + 1) / 2, sms);
  a.part_stride = fp8_part_bytes(a.R) / 4;
  Fp8Maps maps;
  memset(&maps, 0, sizeof maps);
  if (!byte_map(&maps.x, a.xq, a.K, a.n_x, 1, 2, kM) ||
      !byte_map(&maps.w[0], a.wq[0], a.K, a.N, a.E, 3, 128) ||
      (SWIGLU && !byte_map(&maps.w[1], a.wq[1], a.K, a.N, a.E, 3, 128)))
    return cudaErrorInvalidValue;
  if (!SWIGLU) maps.w[1] = maps.w[0];
  // 32-byte stores: whole groups of 32 bytes inside every row
  const uint32_t group = 32 / (SWIGLU ? 1 : (uint32_t)dtype_size(a.odt));
  const bool vec = ((uintptr_t)a.out & 31) == 0 && a.N % group == 0 && a.ld % group == 0;
  auto kern = k_fp8_tc<SWIGLU>;
  const size_t rest = 1024 + 512 + 2048 + 4 * kScaleSlots * (kM + 2) + fp8_tiles_smem(a.E);
  int ns = (int)((kSmemLimit - rest) / kStage);
  if (ns > (int)kTcStages) ns = kTcStages;
  const size_t smem = rest + ns * (size_t)kStage;
  static std::atomic<bool> done[kMaxDevices];
  const cudaError_t e = allow_smem(kern, done);
  if (e != cudaSuccess) return e;
  return launch_k(kern, sms, kTcThreads, smem, stream, true, a, maps, (uint32_t)ns, vec);
}

}  // namespace

bool fp8_tc_ok(const Fp8Args &a) {
  auto a16 = [](const void *p) { return ((uintptr_t)p & 15) == 0; };
  return a.K % 16 == 0 && a16(a.xq) && a16(a.wq[0]) && a16(a.wq[1]) && encode_fn() != nullptr;
}

size_t fp8_part_bytes(uint32_t rows) {
  // 256 columns of fp32 for each row of the largest tile that a call of so many rows
  // can take: the few-row kernels' 32 or 64, the many-row kernel's 128 in runs of 32
  const uint32_t r = rows <= kFp8FewProduct32 ? 32
                     : rows <= 64             ? 64
                     : rows < 128             ? (rows + 31) / 32 * 32
                                              : 128;
  return (size_t)r * 1024;
}

size_t fp8_tc_ws(uint32_t rows) { return (size_t)fp8_ctas() * 2 * fp8_part_bytes(rows); }

cudaError_t launch_fp8_tc(Fp8Args &a, bool swiglu, cudaStream_t stream) {
  return swiglu ? run_tc<true>(a, stream) : run_tc<false>(a, stream);
}

}  // namespace moe
