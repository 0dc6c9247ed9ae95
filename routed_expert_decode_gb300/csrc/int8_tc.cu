// int8_tc.cu -- routed and dense products over int8 operands on the 5th-generation tensor
// cores.
//
// The card's integer tensor rate is far below its 16-bit one, so the codes are turned to
// fp16, which holds them exactly, on their way to the MMA (kind::f16, fp32 sums: exact
// while no partial sum passes 2^24; its additions cut off, and odd products of one sign came
// out 3.4e-5 low for K 8208, 8.7e-4 for 131056).  A byte b of b ^ 0x80 under the high byte 0x64 is
// the fp16 number 1024 + 128 + code; a subtraction of 1152 leaves the code: five
// instructions for four codes.
//
// A tile is 128 weight rows (128 channels, or 64 gate and 64 up rows of the same features)
// by up to NT activation rows of one expert.  The weights sit on the MMA's M side: they
// come as bytes by TMA, and the converting warps write them to TMEM, from where the MMA
// takes its A operand, so that they cross shared memory once, as bytes.  The activation
// rows are the N side: the converting warps fetch their bytes through perm straight to
// registers, a block of 128 codes ahead, and store fp16 in the swizzled layout.  The MMA's
// N is the tile's rows rounded up to 16.
//
// Experts with many rows: two CTAs work on a tile of 256 weight rows (cta_group::2), each
// with its own 128 in its TMEM and half of the activation rows in its shared memory.  One
// CTA's N side alone, fp16 written and read again, is all that its shared memory can move
// while the tensor cores work (128 bytes a clock), and the fetches come on top: 16384 rows
// of gate/up (d 6144, f 2048, 16 experts) take 770 us so, 525 in pairs (1.57 PFLOP/s; 470
// without the activations' conversion, 480 without the epilogue).  The first CTA issues; what it has to know of the second
// one's warps goes over four relaying warps there, because an arrival that makes the work
// behind it visible to the other CTA takes ~800 clocks: with one warp for it 976 us, with the
// converting warps making theirs 1390.
//
// TMEM lane 32q + i is a weight row; for SwiGLU lanes i < 16 of a quarter hold gate rows
// and the others the up rows of the same 16 features, so that g and u meet by one
// shuffle for two activation rows.
//
// Loads of the activations take whole lines, eight lanes a row, and may stay in L1: 64
// bytes a row and step, past L1, cost 1080 us in place of 790 (with one CTA a tile).
//
// Warps: 0 weights by TMA, 1 TMEM owner and MMA issuer, then the weight converters (sets of
// four), the epilogue's, the activation converters and the relays.  The work goes out
// over one CTA (or pair) per SM as Walk says; the shares of a split tile meet in the
// workspace, where the last to arrive adds all of them in order.
#include <string.h>

#include "fp8_tc_ptx.cuh"
#include "int8.cuh"

namespace moe {
namespace {

constexpr uint32_t kRing = 12;    // stages of a ring, at most
constexpr uint32_t kCtrl = 1024;  // bytes for barriers
static_assert((2 * kMaxStages + 2 * kRing + 2 * 8 + 2) * 8 + 12 <= kCtrl, "");

// NT: rows of a tile.  PAIR: a tile of twice the weight rows by two CTAs (cta_group::2), each
// with its own weight rows in its TMEM and half of the activation rows in its shared memory.
template <int NT, bool PAIR>
struct Shape {
  // stages of 64 along K: 32 TMEM columns of weights each; accumulators take the others
  static constexpr uint32_t ring = NT == 32 ? 10 : 8;
  static constexpr uint32_t a_column = 512 - ring * 32;      // first TMEM column of the weights
  static constexpr uint32_t accs = a_column / NT < 8 ? a_column / NT : 8;
  static constexpr int rows = PAIR ? NT / 2 : NT;            // activation rows of a CTA
  static constexpr uint32_t x_bytes = rows * 128;            // ... and their bytes in a stage
  static constexpr int epi = NT >= 128 ? 8 : 4;              // epilogue warps
  static constexpr int w_sets = NT >= 128 ? 1 : 2;           // sets of weight converters, 1 or 2
  static constexpr int x_warps = NT == 32 ? 2 : rows / 32;   // activation converters of a set
  static constexpr int passes = rows / (x_warps * 4);        // rows of a converting lane
  static constexpr int sets = NT >= 128 ? 2 : (int)ring / 2;  // sets of them
  static constexpr int epi0 = 2 + 4 * w_sets, x0 = epi0 + epi;  // first warps
  static constexpr int relay0 = x0 + sets * x_warps;          // a pair's relaying warps
  static constexpr int relays = PAIR ? 4 : 0;
  static constexpr int threads = (relay0 + relays) * 32;
  static constexpr int cols = NT / (epi / 4);                // columns of an epilogue warp
  static constexpr bool split = NT == 32;                    // tiles may be shared along K
  static constexpr int ctas = PAIR ? 2 : 1;
  static_assert(sets <= (int)ring / 2 && cols % 32 == 0, "");
};

// 16 bytes that other loads of this SM may want again.  Volatile, as ld_once16.
__device__ __forceinline__ uint4 ld_again16(const void *p) {
  uint4 w;
  asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "l"(p));
  return w;
}
// four codes to fp16
__device__ __forceinline__ void i8x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  const uint32_t u = w ^ 0x80808080u;
  const uint32_t bias = 0x64806480u;  // 1152, twice
  uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 c = *reinterpret_cast<const __half2 *>(&bias);
  const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), c);
  const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), c);
  lo = *reinterpret_cast<const uint32_t *>(&x);
  hi = *reinterpret_cast<const uint32_t *>(&y);
}

// 32 columns of this warp's 32 TMEM lanes
__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// D (+)= A B^T over 64 codes of K: four MMAs of K = 16, 8 TMEM columns of A and 32 bytes of
// B's rows apart.  Called by a whole converged warp with uniform operands; one lane issues.
template <bool PAIR>
__device__ __forceinline__ void tc_mma_step(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            bool add) {
  if (PAIR)
    asm volatile(
        "{\n .reg .pred e, f, t;\n .reg .b64 b1, b2, b3;\n .reg .b32 a1, a2, a3;\n"
        " add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"
        " add.u32 a1, %1, 8;\n add.u32 a2, %1, 16;\n add.u32 a3, %1, 24;\n"
        " setp.ne.b32 f, %4, 0;\n setp.eq.b32 t, 0, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, f;\n"
        " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [a1], b1, %3, t;\n"
        " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [a2], b2, %3, t;\n"
        " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [a3], b3, %3, t;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred e, f, t;\n .reg .b64 b1, b2, b3;\n .reg .b32 a1, a2, a3;\n"
        " add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"
        " add.u32 a1, %1, 8;\n add.u32 a2, %1, 16;\n add.u32 a3, %1, 24;\n"
        " setp.ne.b32 f, %4, 0;\n setp.eq.b32 t, 0, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// arrive on the barrier (PAIR: of the CTAs in the mask) when the MMAs so far are done
template <bool PAIR>
__device__ __forceinline__ void tc_commit_all(uint64_t *bar, uint16_t ctas = 3) {
  if (!PAIR) return tc_commit(bar);
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;\n}\n" ::"r"(s32(bar)),
      "h"(ctas)
      : "memory");
}
// the first CTA's barrier at this place, as an address of the pair
__device__ __forceinline__ uint32_t leader_bar(uint64_t *b) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(s32(b)));
  return r;
}
// one arrival on the barrier that the MMA's issuer waits on
template <bool PAIR>
__device__ __forceinline__ void arrive_issuer(uint64_t *b) {
  if (!PAIR) return bar_arrive(b);
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_bar(b))
               : "memory");
}
// bar_wait for arrivals of both CTAs
__device__ __forceinline__ bool pair_try(uint64_t *b, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(s32(b)), "r"(parity), "n"(kHintNs)
      : "memory");
  return done != 0;
}
template <bool PAIR>
__device__ __forceinline__ void issuer_wait(uint64_t *b, uint32_t parity, const Guard &g) {
  if (!PAIR) return bar_wait(b, parity, g);
  if (pair_try(b, parity) || *g.abort_flag) return;
  const long long t0 = clock64();
  for (int i = 0; i < kSpin && !*g.abort_flag; ++i) {
    if (pair_try(b, parity)) return;
    if (clock64() - t0 > kWaitCycles) break;
  }
  if (!*g.abort_flag) atomicOr(g.err, kErrTimeout);
  *g.abort_flag = 1;
}
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}

// a place in a ring that is passed `step` stages at a time
template <int STEP>
struct StepRing {
  uint32_t i, phase = 0;
  __device__ __forceinline__ explicit StepRing(uint32_t first) : i(first) {}
  __device__ __forceinline__ void next(uint32_t n) {
    i += STEP;
    if (i >= n) {
      i -= n;
      phase ^= 1;
    }
  }
};

template <bool SWIGLU, int NT, bool PAIR>
__global__ void __launch_bounds__(Shape<NT, PAIR>::threads, 1)
    k_int8_tc(const Fp8Args a, const __grid_constant__ Fp8Maps maps, const uint32_t n_w,
              const int split_below, const int tile_rows, const bool pairs) {
  pdl_trigger();
  using S = Shape<NT, PAIR>;
  extern __shared__ __align__(1024) uint8_t tsm_raw[];
  uint8_t *tsm = tsm_raw + ((0u - s32(tsm_raw)) & 1023u);  // stays a shared address
  const int tid = threadIdx.x, lane = tid & 31;
  // through a shuffle, so that the roles' branches are known to be uniform
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  uint8_t *xsm = tsm + n_w * kWBytes;
  uint8_t *ctrl = xsm + S::ring * S::x_bytes;
  uint64_t *w_full = (uint64_t *)ctrl;     // [kMaxStages] weight bytes of a stage landed
  uint64_t *w_empty = w_full + kMaxStages;  // [kMaxStages] ... read
  uint64_t *full = w_empty + kMaxStages;   // [kRing] a step's operands written
  uint64_t *empty = full + kRing;          // [kRing] ... consumed
  uint64_t *d_full = empty + kRing;           // [8] accumulator written
  uint64_t *d_empty = d_full + 8;          // [8] ... read
  uint64_t *meet_bar = d_empty + 8;        // the epilogue's warps
  uint64_t *drain = meet_bar + 1;          // the MMAs of an aborted call
  uint32_t *tmem_holder = (uint32_t *)(drain + 1);
  volatile int *abort_flag = (volatile int *)(tmem_holder + 1);
  volatile int *last_part = (volatile int *)(tmem_holder + 2);
  float *xsc = (float *)(ctrl + kCtrl);    // [2][NT] row scales of a tile
  int *tiles_sm = (int *)(xsc + 2 * NT);

  if (tid == 32) {
    prefetch_map(&maps.w[0]);
    if (SWIGLU) prefetch_map(&maps.w[1]);
  }
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      bar_init(&w_full[i], 1);
      bar_init(&w_empty[i], 4 * S::w_sets);
    }
    for (uint32_t i = 0; i < kRing; ++i) {
      bar_init(&full[i], 4 + S::x_warps + (PAIR && !(blockIdx.x & 1)));
      bar_init(&empty[i], 1);
    }
    for (uint32_t i = 0; i < 8; ++i) {
      bar_init(&d_full[i], 1);
      bar_init(&d_empty[i], S::ctas * S::epi);
    }
    bar_init(meet_bar, S::epi);
    bar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    if (PAIR) {
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
  if (PAIR) pair_sync();  // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  fp8_warm(a);
  pdl_wait();
  const RowTiles rt = fp8_row_tiles<NT>(a, tiles_sm, tile_rows);
  const int rank = PAIR ? (int)(blockIdx.x & 1) : 0;
  Walk walk(rt.total * (int)a.n_tiles, a, (int)blockIdx.x / S::ctas, (int)gridDim.x / S::ctas,
            split_below);
  Seg seg;
  const Guard guard{a.err, abort_flag};
  // this CTA's block of weight rows
  auto block_of = [&](const Fp8Tile &t) { return t.nt * S::ctas + rank; };
  // columns of the MMA: the tile's rows, rounded up so that each CTA has a multiple of 16
  auto mma_rows = [](int rows) { return PAIR ? (rows + 31) & ~31 : (rows + 15) & ~15; };

  if (warp == 0) {
    // ============================ weights
    Ring st;
    while (!guard.aborted() && walk.take(seg)) {
      const Fp8Tile t = fp8_tile<NT>(a, rt, seg.tile, tile_rows);
      for (int kb = seg.kb0; kb < seg.kb1; ++kb, st.next(n_w)) {
        bar_wait(&w_empty[st.i], st.phase ^ 1, guard);  // the first use passes
        __syncwarp();
        if (guard.aborted()) break;
        if (lane) continue;
        uint8_t *dst = tsm + st.i * kWBytes;
        bar_expect(&w_full[st.i], kWBytes);
        if (SWIGLU) {
          tma_w(dst, &maps.w[0], kb * 128, block_of(t) * 64, t.e, &w_full[st.i]);
          tma_w(dst + kWBytes / 2, &maps.w[1], kb * 128, block_of(t) * 64, t.e, &w_full[st.i]);
        } else {
          tma_w(dst, &maps.w[0], kb * 128, block_of(t) * 128, t.e, &w_full[st.i]);
        }
      }
    }
    // the stages still in use: leave with no copy in flight
    for (uint32_t i = 0; i < n_w; ++i, st.next(n_w))
      if (!bar_wait_for(*abort_flag ? &w_full[st.i] : &w_empty[st.i], st.phase ^ 1))
        atomicOr(a.err, kErrTimeout);
  } else if (warp == 1) {
    // ============================ MMA issuer (of a pair, the first CTA's)
    Ring st, acc;
    while (!guard.aborted() && walk.take(seg)) {
      const int steps = 2 * (seg.kb1 - seg.kb0);
      if (PAIR && rank) {  // follows the ring, for its end
        for (int s = 0; s < steps; ++s) st.next(S::ring);
        continue;
      }
      const Fp8Tile t = fp8_tile<NT>(a, rt, seg.tile, tile_rows);
      // M = 128, or 256 of a pair
      const uint32_t idesc = idesc_for((uint32_t)mma_rows(t.rows)) + (PAIR ? 8u << 24 : 0u);
      const uint32_t d = tmem + acc.i * NT;
      issuer_wait<PAIR>(&d_empty[acc.i], acc.phase ^ 1, guard);
      for (int s = 0; s < steps; ++s, st.next(S::ring)) {
        issuer_wait<PAIR>(&full[st.i], st.phase, guard);
        tc_fence_after();
        __syncwarp();
        tc_mma_step<PAIR>(d, tmem + S::a_column + st.i * 32,
                          sw128_desc(s32(xsm + st.i * S::x_bytes)), idesc, s > 0);
        tc_commit_all<PAIR>(&empty[st.i]);
      }
      tc_commit_all<PAIR>(&d_full[acc.i]);
      acc.next(S::accs);
    }
    if (guard.aborted()) {
      if (!rank) {
        tc_commit_all<PAIR>(drain, 1);
        bar_wait_for(drain, 0);
      }
    } else {  // the last steps' arrivals
      for (uint32_t i = 0; i < S::ring; ++i, st.next(S::ring))
        if (!bar_wait_for(&empty[st.i], st.phase ^ 1)) atomicOr(a.err, kErrTimeout);
    }
  } else if (warp < S::epi0) {
    // ============================ weight converters: half `set` of each stage
    const int set = (warp - 2) >> 2, quarter = warp & 3;
    const int row = SWIGLU ? quarter * 16 + (lane & 15) + (lane >> 4) * 64 : quarter * 32 + lane;
    const uint32_t dst = tmem + S::a_column + ((uint32_t)(quarter * 32) << 16);
    Ring ws, st;  // st: of pairs of steps
    while (!guard.aborted() && walk.take(seg)) {
      for (int kb = seg.kb0; kb < seg.kb1; ++kb, ws.next(n_w), st.next(S::ring / 2)) {
        bar_wait(&w_full[ws.i], ws.phase, guard);
        // 128-byte swizzle: chunk c of row r at c ^ (r % 8)
        const uint8_t *src = tsm + ws.i * kWBytes + row * 128;
#pragma unroll
        for (int h0 = 0; h0 < 2; h0 += S::w_sets) {
          const int h = S::w_sets == 2 ? set : h0;
          const uint32_t stage = 2 * st.i + h;
          uint4 v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            v[c] = *(const uint4 *)(src + (((h * 4 + c) ^ (row & 7)) << 4));
          if (h0 + S::w_sets == 2) {
            __syncwarp();
            if (lane == 0) bar_arrive(&w_empty[ws.i]);
          }
          uint32_t r[32];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            i8x4_to_f16(v[c].x, r[8 * c], r[8 * c + 1]);
            i8x4_to_f16(v[c].y, r[8 * c + 2], r[8 * c + 3]);
            i8x4_to_f16(v[c].z, r[8 * c + 4], r[8 * c + 5]);
            i8x4_to_f16(v[c].w, r[8 * c + 6], r[8 * c + 7]);
          }
          bar_wait(&empty[stage], st.phase ^ 1, guard);
          tc_fence_after();
          __syncwarp();
          tc_st32(dst + stage * 32, r);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          tc_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&full[stage]);
        }
      }
    }
  } else if (warp < S::x0) {
    // ============================ epilogue
    const int ew = warp - S::epi0, quarter = warp & 3, c0 = (ew >> 2) * S::cols;
    Ring dr;
    uint32_t nmeet = 0, tiles = 0;
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) bar_arrive(meet_bar);
      bar_wait(meet_bar, nmeet++ & 1, guard);
      __syncwarp();
    };
    while (!guard.aborted() && walk.take(seg)) {
      const Fp8Tile t = fp8_tile<NT>(a, rt, seg.tile, tile_rows);
      // ---- scales: one a row through shared memory, one a lane
      float *xs = xsc + (tiles++ & 1) * NT;
      for (int r = ew * 32 + lane; r < t.rows; r += S::epi * 32)
        xs[r] = a.xs[max(0, fp8_x_row(a, t.row0 + r))];
      const uint32_t n = SWIGLU ? (uint32_t)block_of(t) * 64 + quarter * 16 + (lane & 15)
                                : (uint32_t)block_of(t) * 128 + quarter * 32 + lane;
      const bool up = SWIGLU && lane >= 16;
      const float ws = n < a.N ? a.wsc[up ? 1 : 0][(size_t)t.e * a.N + n] : 0.0f;
      meet();
      const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + dr.i * NT + c0;
      // columns c .. c + 31 of the tile, as sums in v, to the outputs
      auto emit = [&](int c, const float (&v)[32]) {
        const int rows = t.rows - c;
        float s[32];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 x = *(const float4 *)(xs + c + i);
          s[i] = v[i] * (x.x * ws);
          s[i + 1] = v[i + 1] * (x.y * ws);
          s[i + 2] = v[i + 2] * (x.z * ws);
          s[i + 3] = v[i + 3] * (x.w * ws);
        }
        // SwiGLU: lanes of gate rows take row i0 + 2i, those of up rows the next
        auto swiglu8 = [&](int i0, float (&h)[4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = s[i0 + 2 * i], y = s[i0 + 2 * i + 1];
            const float got = __shfl_xor_sync(0xffffffffu, up ? x : y, 16);
            h[i] = fp8_swiglu_value(up ? got : x, up ? y : got);
          }
        };
        // eight rows at a time without a branch between them: their latencies overlap
        auto store = [&](auto *p, auto from) {
          p += (size_t)(t.row0 + c) * a.ld + n;
#pragma unroll
          for (int i0 = 0; i0 < 32; i0 += 8) {
            if (i0 >= rows) break;  // the warp alike
            if (!SWIGLU) {
#pragma unroll
              for (int i = i0; i < i0 + 8; ++i)
                if (n < a.N && i < rows) p[(size_t)i * a.ld] = from(s[i]);
            } else {
              float h[4];
              swiglu8(i0, h);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = i0 + 2 * i + up;
                if (n < a.N && r < rows) p[(size_t)r * a.ld] = from(h[i]);
              }
            }
          }
        };
        // 16-bit types, two channels a store: a lane pair's even lane takes the first of two
        // values, the odd lane the second
        auto store2 = [&](auto pack) {
          const bool odd = lane & 1;
          uint16_t *p = (uint16_t *)a.out + (size_t)(t.row0 + c) * a.ld + (n & ~1u);
          auto two = [&](float first, float second, int r0, int r1) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? first : second, 1);
            const uint32_t w = odd ? pack(got, second) : pack(first, got);
            const int r = odd ? r1 : r0;
            if (n < a.N && r < rows) *(uint32_t *)(p + (size_t)r * a.ld) = w;
          };
#pragma unroll
          for (int i0 = 0; i0 < 32; i0 += 8) {
            if (i0 >= rows) break;  // the warp alike
            if (!SWIGLU) {
#pragma unroll
              for (int i = i0; i < i0 + 8; i += 2) two(s[i], s[i + 1], i, i + 1);
            } else {
              float h[4];
              swiglu8(i0, h);
              two(h[0], h[1], i0 + up, i0 + 2 + up);
              two(h[2], h[3], i0 + 4 + up, i0 + 6 + up);
            }
          }
        };
        if (a.odt == MOE_DT_F32) store((float *)a.out, [](float x) { return x; });
        else if (a.odt == MOE_DT_BF16 && pairs) store2(pack2<MOE_DT_BF16>);
        else if (pairs) store2(pack2<MOE_DT_F16>);
        else if (a.odt == MOE_DT_BF16) store((__nv_bfloat16 *)a.out, Elem<MOE_DT_BF16>::from);
        else store((__half *)a.out, Elem<MOE_DT_F16>::from);
      };
      const bool whole = seg.kb1 - seg.kb0 == (int)a.nbk;
      bar_wait(&d_full[dr.i], dr.phase, guard);
      tc_fence_after();
      __syncwarp();
      if (!S::split || whole) {
#pragma unroll 1
        for (int c = 0; c < S::cols; c += 32) {
          if (c0 + c >= t.rows) break;
          float v[32];
          tc_ld32(src + c, v);
          tc_wait_ld32(v);
          if (c + 32 >= S::cols || c0 + c + 32 >= t.rows) {  // the last of this warp's
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_issuer<PAIR>(&d_empty[dr.i]);
          }
          emit(c0 + c, v);
        }
        if (c0 >= t.rows && lane == 0) arrive_issuer<PAIR>(&d_empty[dr.i]);
        dr.next(S::accs);
        continue;
      }
      // ---- a share of a tile: the last of its workers adds up all shares
      const int w0 = walk.first_worker(seg.tile);
      const int shares = walk.last_worker(seg.tile) - w0 + 1;
      // part of worker w: its second slot if it starts the tile, its first otherwise
      auto part = [&](int w, int c) {
        return a.part + (size_t)(2 * w + (w == w0)) * a.part_stride + (size_t)c * 128 +
               quarter * 32 + lane;
      };
#pragma unroll 1
      for (int c = 0; c < S::cols && c < t.rows; c += 32) {
        float v[32];
        tc_ld32(src + c, v);
        tc_wait_ld32(v);
        float *mine = part((int)blockIdx.x, c);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c + i < t.rows) __stcg(mine + i * 128, v[i]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_issuer<PAIR>(&d_empty[dr.i]);
      dr.next(S::accs);
      __threadfence();
      meet();
      if (ew == 0 && lane == 0) {
        __threadfence();
        uint32_t *count = a.sync + 4 * seg.tile;
        const bool last = atomicAdd(count, 1u) == (uint32_t)shares - 1;
        if (last) atomicExch(count, 0u);
        *last_part = last;
      }
      meet();
      if (!*last_part) continue;
      __threadfence();
#pragma unroll 1
      for (int c = 0; c < S::cols && c < t.rows; c += 32) {
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.0f;
#pragma unroll 2
        for (int p = 0; p < shares; ++p) {
          const float *q = part(w0 + p, c);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i < t.rows) v[i] += __ldcg(q + i * 128);
        }
        emit(c, v);
      }
    }
  } else if (PAIR && warp >= S::relay0) {
    // ============================ relay: passes the second CTA's arrivals on to the issuer.
    // Such an arrival makes all that it follows visible to the other CTA, ~800 clocks
    // each: several are on the way together.
    StepRing<PAIR ? S::relays : 1> st(warp - S::relay0);
    int first = warp - S::relay0;
    while (rank && !guard.aborted() && walk.take(seg)) {
      const int steps = 2 * (seg.kb1 - seg.kb0);
      for (int s = first; s < steps; s += PAIR ? S::relays : 1, st.next(S::ring)) {
        bar_wait(&full[st.i], st.phase, guard);
        __syncwarp();
        if (lane == 0) arrive_issuer<true>(&full[st.i]);
      }
      first = (first - steps % (PAIR ? S::relays : 1) + S::relays) % (PAIR ? S::relays : 1);
    }
  } else {
    // ============================ activation converters: eight lanes a row of 128 codes, the
    // first four of which write a block's first step and the others its second
    const int xw = warp - S::x0, set = xw / S::x_warps;
    const int th = (xw - set * S::x_warps) * 32 + lane, chunk = th & 7, r0 = th >> 3;
    const int step = chunk >> 2, c0 = 2 * (chunk & 3);  // 16-byte chunks c0, c0 + 1 of fp16
    constexpr int kPass = S::x_warps * 4, kPasses = S::passes;  // rows of a pass over the set's threads
    constexpr uint32_t kBlocks = S::ring / 2;
    StepRing<S::sets> st(set);
    int first = set;  // this set's first block of the segment
    while (!guard.aborted() && walk.take(seg)) {
      const Fp8Tile t = fp8_tile<NT>(a, rt, seg.tile, tile_rows);
      const int rows = mma_rows(t.rows) / S::ctas;  // this CTA's
      int row[kPasses];  // a bad one (flagged) reads row 0
#pragma unroll
      for (int j = 0; j < kPasses; ++j) {
        const int r = rank * rows + r0 + j * kPass;
        row[j] = r0 + j * kPass < rows && r < t.rows ? max(0, fp8_x_row(a, t.row0 + r)) : -1;
      }
      uint4 v[kPasses];
      auto load = [&](int kb) {
        const uint32_t k = (uint32_t)kb * 128 + chunk * 16;
#pragma unroll
        for (int j = 0; j < kPasses; ++j) {
          v[j] = make_uint4(0, 0, 0, 0);
          if (kb < seg.kb1 && row[j] >= 0 && k < a.K)
            v[j] = ld_again16(a.xq + (size_t)(uint32_t)row[j] * a.K + k);
        }
      };
      load(seg.kb0 + first);
      for (int kb = seg.kb0 + first; kb < seg.kb1; kb += S::sets) {
        bar_wait(&empty[2 * st.i], st.phase ^ 1, guard);
        bar_wait(&empty[2 * st.i + 1], st.phase ^ 1, guard);
        const uint32_t buf = s32(xsm + (2 * st.i + step) * S::x_bytes);
#pragma unroll
        for (int j = 0; j < kPasses; ++j) {
          const int r = r0 + j * kPass;
          if (r >= rows) break;
          uint32_t h[8];
          i8x4_to_f16(v[j].x, h[0], h[1]);
          i8x4_to_f16(v[j].y, h[2], h[3]);
          i8x4_to_f16(v[j].z, h[4], h[5]);
          i8x4_to_f16(v[j].w, h[6], h[7]);
          // 128-byte swizzle: chunk c of row r at c ^ (r % 8).  The second step's lanes
          // store their second chunk first, so that eight lanes meet all banks.
          const uint32_t at = buf + r * 128;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const bool second = q != step;
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                             at + (((c0 + second) ^ (r & 7)) << 4)),
                         "r"(second ? h[4] : h[0]), "r"(second ? h[5] : h[1]),
                         "r"(second ? h[6] : h[2]), "r"(second ? h[7] : h[3])
                         : "memory");
          }
        }
        fence_async();  // read by the tensor core's proxy
        __syncwarp();
        if (lane < 2) bar_arrive(&full[2 * st.i + lane]);
        st.next(kBlocks);
        load(kb + S::sets);
      }
      first = (first - (seg.kb1 - seg.kb0) % S::sets + S::sets) % S::sets;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) pair_sync();  // neither CTA leaves while the other may reach its memory
  if (warp == 1) {
    tc_fence_after();
    if (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// What the tiles take by the rows of an expert, on average: 32 experts, gate/up 4096 -> 2 x 2048
// and down 2048 -> 4096, a router's spread of rows (us):
//   rows            8        16        32        64        96       128       192       512
//   tile  32    87  49   95  53   116  65   189 105   264 146   335 185   480 263  1208 659
//         64    88  50   92  53   107  62   137  80   184 107   230 133   320 185   760 440
//        128   106  57  109  58   115  63   143  78   168  92   194 105   270 145   594 316
//   256 pair   145  78  146  79   150  83   157  90   171 100   187 113   217 133   427 256
//
// The choice goes by a sum of what these and calls of fewer tiles measured: a call takes a
// fixed time and, for each round of tiles over the SMs (pairs), so much a step of 64 along K
// and a tile's end.  One expert's rows are known here, and its rounds counted; its pairs' tiles
// are cut to a height that fills the last round (4000 rows, 4096 channels: 18 of 224 rows).  Of
// several experts the average is: each has half a tile more than its share of the rows, and
// some have two where that is about one.
// 24 experts of 351 rows, K 3328, f 176: 38 us, 47 with the tile by rows alone; 4 of 1550, K
// 2592, 128 channels: 15 and 25.
struct Plan {
  int tile = 0, rows = 0;  // NT (256: pairs) and the rows of a tile
  Plan(const Fp8Args &a, bool swiglu, int sms) {
    const double steps = (a.K + 63) / 64, R = a.R, live = a.R < a.E ? a.R : a.E;
    double least = 1e30;
    auto take = [&](int nt, int height, uint32_t columns, int workers, double fixed, double step,
                    double end) {
      double each = 1;  // tiles of an expert's rows
      if (a.E == 1) {
        each = (a.R + height - 1) / height;
      } else {
        const double full = R / (live * height);
        if (0.75 + 0.75 * full > each) each = 0.75 + 0.75 * full;
        if (full + 0.5 > each) each = full + 0.5;
      }
      const double tiles = live * each * ((a.N + columns - 1) / columns);
      const double x = tiles / workers;
      const double rounds = x <= 1 ? 1 : x < 3 ? (double)(int)(x + 0.999) : x + 0.5;
      double us = fixed + rounds * (steps * step + end);
      // a last round shared along K (run_tc)
      if (nt == 32 && x < split_share((uint32_t)steps) && us > fixed + x * steps * step + 9.5)
        us = fixed + x * steps * step + 9.5;
      if (us < least) {
        least = us;
        tile = nt;
        rows = height;
      }
    };
    const uint32_t channels = swiglu ? 64 : 128;
    take(32, 32, channels, sms, 4.2, 0.185, 0.5);
    take(64, 64, channels, sms, 4.6, 0.20, 0.5);
    take(128, 128, channels, sms, 4.5, 0.30, 0.3);
    if (sms > 1)
      for (int h = 256; h >= (a.E == 1 ? 128 : 256); h -= 32)
        take(256, h, 2 * channels, sms / 2, 3.5, 0.35 * (h + 24) / 280, 3.5);
  }
  // A last round of fewer tiles than this part of the SMs is shared along K: a meeting costs
  // ~9.5 us, the time of some 55 steps (16 rows, 4096 channels, K 6144: 16.9 us, 20 whole; 128
  // rows, 1024 features, K 4096: 18.6 and 15.8).
  static double split_share(uint32_t steps) { return steps > 55 ? 1.0 - 55.0 / steps : 0.0; }
};

template <bool SWIGLU, int NT, bool PAIR>
cudaError_t run_tc(Fp8Args &a, cudaStream_t stream, int tile_rows = NT) {
  using S = Shape<NT, PAIR>;
  const int sms = fp8_ctas() / S::ctas * S::ctas;
  if (sms < S::ctas) return cudaErrorInvalidValue;
  const uint32_t channels = SWIGLU ? 64 : 128;  // of a CTA
  fp8_set_tiles(a, (a.N + channels * S::ctas - 1) / (channels * S::ctas), sms / S::ctas);
  a.part_stride = (size_t)NT * 128;
  Fp8Maps maps;
  memset(&maps, 0, sizeof maps);
  for (int m = 0; m < (SWIGLU ? 2 : 1); ++m)
    if (!byte_map(&maps.w[m], a.wq[m], a.K, a.N, a.E, 3, channels)) return cudaErrorInvalidValue;
  auto kern = k_int8_tc<SWIGLU, NT, PAIR>;
  const size_t rest =
      1024 + S::ring * (size_t)S::x_bytes + kCtrl + 4 * 2 * NT + fp8_tiles_smem(a.E);
  int n_w = (int)((kSmemLimit - rest) / kWBytes);
  if (n_w > kMaxStages) n_w = kMaxStages;
  const size_t smem = rest + (size_t)n_w * kWBytes;
  static std::atomic<bool> done[kMaxDevices];
  const cudaError_t e = allow_smem(kern, done);
  if (e != cudaSuccess) return e;
  const int split_below = S::split ? (int)(sms * Plan::split_share(2 * a.nbk)) : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = sms;
  cfg.blockDim = S::threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {2, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  const bool pairs = ((uintptr_t)a.out & 3) == 0 && a.ld % 2 == 0 && a.N % 2 == 0;
  return cudaLaunchKernelEx(&cfg, kern, a, maps, (uint32_t)n_w, split_below, tile_rows, pairs);
}

template <bool SWIGLU>
cudaError_t run_planned(Fp8Args &a, cudaStream_t stream) {
  const Plan plan(a, SWIGLU, fp8_ctas());
  if (plan.tile == 32) return run_tc<SWIGLU, 32, false>(a, stream);
  if (plan.tile == 64) return run_tc<SWIGLU, 64, false>(a, stream);
  if (plan.tile == 128) return run_tc<SWIGLU, 128, false>(a, stream);
  return run_tc<SWIGLU, 256, true>(a, stream, plan.rows);
}

}  // namespace

bool int8_tc_ok(const Fp8Args &a) {
  auto a16 = [](const void *p) { return ((uintptr_t)p & 15) == 0; };
  return a.K % 16 == 0 && a16(a.xq) && a16(a.wq[0]) && a16(a.wq[1]) && encode_fn() != nullptr;
}

// two shares a CTA of a tile of 32 rows
size_t int8_tc_ws() { return (size_t)fp8_ctas() * 2 * 32 * 128 * 4; }

cudaError_t launch_int8_tc(Fp8Args &a, bool swiglu, cudaStream_t stream) {
  return swiglu ? run_planned<true>(a, stream) : run_planned<false>(a, stream);
}

}  // namespace moe
