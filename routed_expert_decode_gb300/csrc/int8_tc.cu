// int8_tc.cu -- routed and dense products over int8 operands on the 5th-generation tensor
// cores.
//
// The card's integer tensor rate is far below its 16-bit one, so the codes are turned to
// fp16, which holds them exactly, on their way to the MMA (kind::f16, fp32 sums: exact
// while no partial sum passes 2^24).  A byte b of b ^ 0x80 under the high byte 0x64 is
// the fp16 number 1024 + 128 + code; a subtraction of 1152 leaves the code: five
// instructions for four codes.
//
// A tile is 128 weight rows (128 channels, or 64 gate and 64 up rows of the same features)
// by up to NT activation rows of one expert.  The weights sit on the MMA's M side: they
// come as bytes by TMA, and the converting warps write them to TMEM, from where the MMA
// takes its A operand, so that they cross shared memory once, as bytes.  The activation
// rows are the N side: the converting warps fetch their bytes through perm straight to
// registers, two steps of K ahead, and store fp16 in the swizzled layout.  The MMA's N is
// the tile's rows rounded up to 16.
//
// TMEM lane 32q + i is a weight row; for SwiGLU lanes i < 16 of a quarter hold gate rows
// and the others the up rows of the same 16 features, so that g and u meet by one
// shuffle for two activation rows.
//
// Warps: 0 weights by TMA, 1 TMEM owner and MMA issuer, 2..9 weight converters (one set
// of four for each half of a stage's 128 codes), then the epilogue's, then the activation
// converters.  The work goes out over one CTA per SM as Walk says; the shares of a
// split tile meet in the workspace, where the last to arrive adds all of them in order.
#include <string.h>

#include "fp8_tc_ptx.cuh"
#include "int8.cuh"

namespace moe {
namespace {

constexpr uint32_t kAColumn = 256;  // first TMEM column of the weights' ring

template <bool SWIGLU, int NT>
struct Shape {
  static constexpr uint32_t accs = 256 / NT;               // accumulators, NT columns each
  static constexpr uint32_t ring = NT == 256 ? 4 : 8;      // stages of 64 along K
  static constexpr uint32_t x_bytes = NT * 128;            // activations of a stage
  static constexpr int epi = NT >= 128 ? 8 : 4;            // epilogue warps
  static constexpr int sets = NT == 256 ? 1 : 2;           // sets of activation converters
  static constexpr int x_warps = NT / 32;                  // warps of a set
  static constexpr int epi0 = 10, x0 = epi0 + epi;         // first warps
  static constexpr int threads = (x0 + sets * x_warps) * 32;
  static constexpr int cols = NT / (epi / 4);              // columns of an epilogue warp
  static constexpr bool split = NT <= 64;                  // tiles may be shared along K
};

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
__device__ __forceinline__ void tc_mma_step(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            bool add) {
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

template <bool SWIGLU, int NT>
__global__ void __launch_bounds__(Shape<SWIGLU, NT>::threads, 1)
    k_int8_tc(const Fp8Args a, const __grid_constant__ Fp8Maps maps, const uint32_t n_w,
              const int split_below) {
  pdl_trigger();
  using S = Shape<SWIGLU, NT>;
  extern __shared__ __align__(1024) uint8_t tsm_raw[];
  uint8_t *tsm = tsm_raw + ((0u - s32(tsm_raw)) & 1023u);  // stays a shared address
  const int tid = threadIdx.x, lane = tid & 31;
  // through a shuffle, so that the roles' branches are known to be uniform
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  uint8_t *xsm = tsm + n_w * kWBytes;
  uint8_t *ctrl = xsm + S::ring * S::x_bytes;
  uint64_t *w_full = (uint64_t *)ctrl;     // [kMaxStages] weight bytes of a stage landed
  uint64_t *w_empty = w_full + kMaxStages;  // [kMaxStages] ... read
  uint64_t *full = w_empty + kMaxStages;   // [8] a step's operands written
  uint64_t *empty = full + 8;              // [8] ... consumed
  uint64_t *d_full = empty + 8;            // [8] accumulator written
  uint64_t *d_empty = d_full + 8;          // [8] ... read
  uint64_t *meet_bar = d_empty + 8;        // the epilogue's warps
  uint64_t *drain = meet_bar + 1;          // the MMAs of an aborted call
  uint32_t *tmem_holder = (uint32_t *)(drain + 1);
  volatile int *abort_flag = (volatile int *)(tmem_holder + 1);
  volatile int *last_part = (volatile int *)(tmem_holder + 2);
  float *xsc = (float *)(ctrl + 512);      // [2][NT] row scales of a tile
  int *tiles_sm = (int *)(xsc + 2 * NT);

  if (tid == 32) {
    prefetch_map(&maps.w[0]);
    if (SWIGLU) prefetch_map(&maps.w[1]);
  }
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      bar_init(&w_full[i], 1);
      bar_init(&w_empty[i], 8);
    }
    for (uint32_t i = 0; i < 8; ++i) {
      bar_init(&full[i], 4 + S::x_warps);
      bar_init(&empty[i], 1);
      bar_init(&d_full[i], 1);
      bar_init(&d_empty[i], S::epi);
    }
    bar_init(meet_bar, S::epi);
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
  const RowTiles rt = fp8_row_tiles<NT>(a, tiles_sm);
  Walk walk(rt.total * (int)a.n_tiles, a, (int)blockIdx.x, (int)gridDim.x, split_below);
  Seg seg;
  const Guard guard{a.err, abort_flag};

  if (warp == 0) {
    // ============================ weights
    Ring st;
    while (!guard.aborted() && walk.take(seg)) {
      const Fp8Tile t = fp8_tile<NT>(a, rt, seg.tile);
      for (int kb = seg.kb0; kb < seg.kb1; ++kb, st.next(n_w)) {
        bar_wait(&w_empty[st.i], st.phase ^ 1, guard);  // the first use passes
        __syncwarp();
        if (guard.aborted()) break;
        if (lane) continue;
        uint8_t *dst = tsm + st.i * kWBytes;
        bar_expect(&w_full[st.i], kWBytes);
        if (SWIGLU) {
          tma_w(dst, &maps.w[0], kb * 128, t.nt * 64, t.e, &w_full[st.i]);
          tma_w(dst + kWBytes / 2, &maps.w[1], kb * 128, t.nt * 64, t.e, &w_full[st.i]);
        } else {
          tma_w(dst, &maps.w[0], kb * 128, t.nt * 128, t.e, &w_full[st.i]);
        }
      }
    }
    // the stages still in use: leave with no copy in flight
    for (uint32_t i = 0; i < n_w; ++i, st.next(n_w))
      if (!bar_wait_for(*abort_flag ? &w_full[st.i] : &w_empty[st.i], st.phase ^ 1))
        atomicOr(a.err, kErrTimeout);
  } else if (warp == 1) {
    // ============================ MMA issuer
    Ring st, acc;
    while (!guard.aborted() && walk.take(seg)) {
      const Fp8Tile t = fp8_tile<NT>(a, rt, seg.tile);
      const uint32_t idesc = idesc_for((uint32_t)(t.rows + 15) & ~15u);
      const uint32_t d = tmem + acc.i * NT;
      bar_wait(&d_empty[acc.i], acc.phase ^ 1, guard);
      const int steps = 2 * (seg.kb1 - seg.kb0);
      for (int s = 0; s < steps; ++s, st.next(S::ring)) {
        bar_wait(&full[st.i], st.phase, guard);
        tc_fence_after();
        __syncwarp();
        tc_mma_step(d, tmem + kAColumn + st.i * 32, sw128_desc(s32(xsm + st.i * S::x_bytes)),
                    idesc, s > 0);
        tc_commit(&empty[st.i]);
      }
      tc_commit(&d_full[acc.i]);
      acc.next(S::accs);
    }
    if (guard.aborted()) {
      tc_commit(drain);
      bar_wait_for(drain, 0);
    } else {  // the last steps' arrivals
      for (uint32_t i = 0; i < S::ring; ++i, st.next(S::ring))
        if (!bar_wait_for(&empty[st.i], st.phase ^ 1)) atomicOr(a.err, kErrTimeout);
    }
  } else if (warp < S::epi0) {
    // ============================ weight converters: half `set` of each stage
    const int set = (warp - 2) >> 2, quarter = warp & 3;
    const int row = SWIGLU ? quarter * 16 + (lane & 15) + (lane >> 4) * 64 : quarter * 32 + lane;
    const uint32_t dst = tmem + kAColumn + ((uint32_t)(quarter * 32) << 16);
    Ring ws;
    StepRing<2> st(set);
    while (!guard.aborted() && walk.take(seg)) {
      for (int kb = seg.kb0; kb < seg.kb1; ++kb, ws.next(n_w), st.next(S::ring)) {
        bar_wait(&w_full[ws.i], ws.phase, guard);
        // 128-byte swizzle: chunk c of row r at c ^ (r % 8)
        const uint8_t *src = tsm + ws.i * kWBytes + row * 128;
        uint4 v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          v[c] = *(const uint4 *)(src + (((set * 4 + c) ^ (row & 7)) << 4));
        __syncwarp();
        if (lane == 0) bar_arrive(&w_empty[ws.i]);
        uint32_t r[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          i8x4_to_f16(v[c].x, r[8 * c], r[8 * c + 1]);
          i8x4_to_f16(v[c].y, r[8 * c + 2], r[8 * c + 3]);
          i8x4_to_f16(v[c].z, r[8 * c + 4], r[8 * c + 5]);
          i8x4_to_f16(v[c].w, r[8 * c + 6], r[8 * c + 7]);
        }
        bar_wait(&empty[st.i], st.phase ^ 1, guard);
        tc_fence_after();
        __syncwarp();
        tc_st32(dst + st.i * 32, r);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&full[st.i]);
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
      const Fp8Tile t = fp8_tile<NT>(a, rt, seg.tile);
      // ---- scales: one a row through shared memory, one a lane
      float *xs = xsc + (tiles++ & 1) * NT;
      for (int r = ew * 32 + lane; r < t.rows; r += S::epi * 32)
        xs[r] = a.xs[max(0, fp8_x_row(a, t.row0 + r))];
      const uint32_t n = SWIGLU ? (uint32_t)t.nt * 64 + quarter * 16 + (lane & 15)
                                : (uint32_t)t.nt * 128 + quarter * 32 + lane;
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
        auto store = [&](auto *p, auto from) {
          p += (size_t)(t.row0 + c) * a.ld + n;
          if (!SWIGLU) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (i >= rows) break;
              if (n < a.N) p[(size_t)i * a.ld] = from(s[i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              if (i >= rows) break;  // the warp alike
              // lanes of gate rows take row i, those of up rows row i + 1
              const float got = __shfl_xor_sync(0xffffffffu, up ? s[i] : s[i + 1], 16);
              const float h = up ? fp8_swiglu_value(got, s[i + 1]) : fp8_swiglu_value(s[i], got);
              const int r = i + up;
              if (n < a.N && r < rows) p[(size_t)r * a.ld] = from(h);
            }
          }
        };
        if (a.odt == MOE_DT_F32) store((float *)a.out, [](float x) { return x; });
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
            if (lane == 0) bar_arrive(&d_empty[dr.i]);
          }
          emit(c0 + c, v);
        }
        if (c0 >= t.rows && lane == 0) bar_arrive(&d_empty[dr.i]);
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
      if (lane == 0) bar_arrive(&d_empty[dr.i]);
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
  } else {
    // ============================ activation converters: four lanes a row of 64 codes
    const int xw = warp - S::x0, set = xw / S::x_warps;
    const int th = (xw - set * S::x_warps) * 32 + lane, chunk = th & 3, r0 = th >> 2;
    constexpr int kPass = NT / 4;  // rows of a pass over the set's threads
    StepRing<S::sets> st(set);
    while (!guard.aborted() && walk.take(seg)) {
      const Fp8Tile t = fp8_tile<NT>(a, rt, seg.tile);
      const int rows16 = (t.rows + 15) & ~15;
      int row[4];  // a bad one (flagged) reads row 0
#pragma unroll
      for (int j = 0; j < 4; ++j)
        row[j] = r0 + j * kPass < t.rows ? max(0, fp8_x_row(a, t.row0 + r0 + j * kPass)) : -1;
      const uint32_t k0 = (uint32_t)seg.kb0 * 128 + chunk * 16;
      const int steps = 2 * (seg.kb1 - seg.kb0);
      auto load = [&](uint4 (&v)[4], int s) {
        const uint32_t k = k0 + s * 64;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = make_uint4(0, 0, 0, 0);
          if (s < steps && row[j] >= 0 && k < a.K)
            v[j] = ld_once16(a.xq + (size_t)(uint32_t)row[j] * a.K + k);
        }
      };
      auto convert = [&](const uint4 (&v)[4]) {
        bar_wait(&empty[st.i], st.phase ^ 1, guard);
        const uint32_t buf = s32(xsm + st.i * S::x_bytes);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = r0 + j * kPass;
          if (r >= rows16) break;
          uint32_t h[8];
          i8x4_to_f16(v[j].x, h[0], h[1]);
          i8x4_to_f16(v[j].y, h[2], h[3]);
          i8x4_to_f16(v[j].z, h[4], h[5]);
          i8x4_to_f16(v[j].w, h[6], h[7]);
          // 128-byte swizzle: chunk c of row r at c ^ (r % 8)
          const uint32_t at = buf + r * 128;
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                           at + (((2 * chunk) ^ (r & 7)) << 4)),
                       "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                       : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                           at + (((2 * chunk + 1) ^ (r & 7)) << 4)),
                       "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7])
                       : "memory");
        }
        fence_async();  // read by the tensor core's proxy
        __syncwarp();
        if (lane == 0) bar_arrive(&full[st.i]);
        st.next(S::ring);
      };
      uint4 v0[4], v1[4];
      load(v0, set);
      load(v1, set + S::sets);
      for (int s = set; s < steps; s += 2 * S::sets) {
        convert(v0);
        load(v0, s + 2 * S::sets);
        if (s + S::sets < steps) {
          convert(v1);
          load(v1, s + 3 * S::sets);
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

template <bool SWIGLU, int NT>
cudaError_t run_tc(Fp8Args &a, cudaStream_t stream) {
  using S = Shape<SWIGLU, NT>;
  const int sms = fp8_ctas();
  const uint32_t channels = SWIGLU ? 64 : 128;
  fp8_set_tiles(a, (a.N + channels - 1) / channels, sms);
  a.part_stride = (size_t)NT * 128;
  Fp8Maps maps;
  memset(&maps, 0, sizeof maps);
  for (int m = 0; m < (SWIGLU ? 2 : 1); ++m)
    if (!byte_map(&maps.w[m], a.wq[m], a.K, a.N, a.E, 3, channels)) return cudaErrorInvalidValue;
  auto kern = k_int8_tc<SWIGLU, NT>;
  const size_t rest =
      1024 + S::ring * (size_t)S::x_bytes + 512 + 4 * 2 * NT + fp8_tiles_smem(a.E);
  int n_w = (int)((kSmemLimit - rest) / kWBytes);
  if (n_w > kMaxStages) n_w = kMaxStages;
  const size_t smem = rest + (size_t)n_w * kWBytes;
  static std::atomic<bool> done[kMaxDevices];
  const cudaError_t e = allow_smem(kern, done);
  if (e != cudaSuccess) return e;
  return launch_k(kern, sms, S::threads, smem, stream, true, a, maps, (uint32_t)n_w,
                  S::split && a.nbk >= 16 ? sms / 4 : 0);
}

template <bool SWIGLU>
cudaError_t run_by_rows(Fp8Args &a, cudaStream_t stream) {
  const uint64_t R = a.R, E = a.E;
  if (R <= 24 * E) return run_tc<SWIGLU, 32>(a, stream);
  if (R <= 64 * E) return run_tc<SWIGLU, 64>(a, stream);
  if (R <= 128 * E) return run_tc<SWIGLU, 128>(a, stream);
  return run_tc<SWIGLU, 256>(a, stream);
}

}  // namespace

bool int8_tc_ok(const Fp8Args &a) {
  auto a16 = [](const void *p) { return ((uintptr_t)p & 15) == 0; };
  return a.K % 16 == 0 && a16(a.xq) && a16(a.wq[0]) && a16(a.wq[1]) && encode_fn() != nullptr;
}

// two shares a CTA of the largest tile that a call of so many rows may split
size_t int8_tc_ws(uint32_t rows) {
  return (size_t)fp8_ctas() * 2 * (rows <= 24 ? 32 : 64) * 128 * 4;
}

cudaError_t launch_int8_tc(Fp8Args &a, bool swiglu, cudaStream_t stream) {
  return swiglu ? run_by_rows<true>(a, stream) : run_by_rows<false>(a, stream);
}

}  // namespace moe
