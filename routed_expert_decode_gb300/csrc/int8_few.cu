// int8_few.cu -- routed products over int8 operands of a few rows in all (decode steps), on
// CUDA cores: bound by the stream of weights from HBM.
//
// A tile of the tensor-core kernel is 128 weight rows; a token's 8 experts have 256 or 384
// of them for 152 SMs, and the last round is short of work.  Here a warp takes four weight
// rows at a time (two gate and two up rows of the same features) and multiplies them with up
// to four activation rows of their expert: 16 codes a lane and row, four at a time by dp4a,
// summed over the lanes by one integer reduction a result, so that sums are exact.  The
// weights' loads run kDepth steps of 512 codes ahead of their use; the activations, all of
// them, lie in shared memory (read through L1: 4 rows of one expert 16.5 us in place of 11.2).
//
// One token of 8 experts, d 6144, f 2048: gate/up 36 us, 5.6 TB/s, down 21, 4.8; 4 tokens
// 104 and 60, 7.2 and 6.3.  A call's launch and prologue are ~5 us of each.
#include "int8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 4;   // activation rows of a tile
constexpr int kDepth = 4;   // steps on the way (one token: 36 us; 36.4 with 3)

// Weight bytes of a warp's run of consecutive units, about: the runs go round the device's
// warps, so that what is read at a time lies close together (30 experts of 25 MB: 104 us; 137
// with one run a warp, which keeps as many places open as there are warps).
constexpr uint32_t kRunBytes = 24576;

struct Cursor {
  uint32_t u, left, run, jump;  // the unit, units behind it in the run, units of a run
  __device__ __forceinline__ Cursor(uint32_t run_, uint32_t w, uint32_t warps)
      : u(w * run_), left(run_), run(run_), jump((warps - 1) * run_) {}
  __device__ __forceinline__ void next() {
    ++u;
    if (--left == 0) {
      left = run;
      u += jump;
    }
  }
};

__device__ __forceinline__ int dot16(const uint4 &a, const uint4 &b, int c) {
  c = __dp4a((int)a.x, (int)b.x, c);
  c = __dp4a((int)a.y, (int)b.y, c);
  c = __dp4a((int)a.z, (int)b.z, c);
  return __dp4a((int)a.w, (int)b.w, c);
}

template <bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1) k_int8_few(const Fp8Args a) {
  pdl_trigger();
  extern __shared__ __align__(16) uint8_t fsm[];
  fp8_warm(a);
  pdl_wait();
  uint8_t *xsm = fsm;  // [n_x][K]
  const RowTiles rt = fp8_row_tiles<kRows>(a, (int *)(fsm + (size_t)a.n_x * a.K));
  const int lane = threadIdx.x & 31;
  const uint32_t warps = gridDim.x * (kThreads / 32);
  const uint32_t w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const uint32_t per = a.n_tiles;  // units of four weight rows of a row tile
  const uint32_t total = (uint32_t)rt.total * per;
  const uint32_t run = total < warps ? 1u : max(1u, kRunBytes / (4 * a.K));
  Cursor ld(run, w, warps), at(run, w, warps);
  const uint32_t steps = (a.K + 511) / 512;
  // expert of row tile q: the largest e with tile[e] <= q
  auto expert_of = [&](int q) {
    const int E = (int)a.E, each = (E + 31) >> 5, first = lane * each;
    const int run =
        __popc(__ballot_sync(0xffffffffu, first < E && rt.tile[min(first, E)] <= q)) - 1;
    const int e = run * each + lane;
    return run * each - 1 + __popc(__ballot_sync(0xffffffffu, lane < each && e < E &&
                                                                  rt.tile[min(e, E)] <= q));
  };
  // ---- what is loaded: kDepth steps ahead of what is multiplied
  uint32_t lq = ld.u / per, ls = 0;
  int le = ld.u < total ? expert_of((int)lq) : 0;
  const uint8_t *src[2];  // first row of the unit, and of its up rows
  auto unit_src = [&]() {
    const uint32_t n = (ld.u - lq * per) * (SWIGLU ? 2 : 4);
    const size_t at = ((size_t)le * a.N + n) * a.K;
    src[0] = a.wq[0] + at;
    src[1] = SWIGLU ? a.wq[1] + at : src[0];
  };
  unit_src();
  auto load = [&](uint4 (&v)[4]) {
    const uint32_t k = ls * 512 + lane * 16, n = (ld.u - lq * per) * (SWIGLU ? 2 : 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = SWIGLU ? i & 1 : i;
      v[i] = make_uint4(0, 0, 0, 0);
      if (ld.u < total && k < a.K && n + row < a.N)
        v[i] = ld_once16(src[SWIGLU ? i >> 1 : 0] + (size_t)row * a.K + k);
    }
    if (ld.u < total && ++ls == steps) {
      ls = 0;
      ld.next();
      if (ld.u < total) {
        if (ld.u - lq * per >= per) {
          lq = ld.u / per;
          le = expert_of((int)lq);
        }
        unit_src();
      }
    }
  };
  uint4 buf[kDepth][4];
#pragma unroll
  for (int i = 0; i < kDepth; ++i) load(buf[i]);
  // ---- the activations, with the first weights on their way
  {
    const uint32_t n16 = (uint32_t)((size_t)a.n_x * a.K / 16);
    for (uint32_t i = threadIdx.x; i < n16; i += kThreads)
      ((uint4 *)xsm)[i] = ld_once16((const uint4 *)a.xq + i);
  }
  __syncthreads();
  // ---- what is multiplied
  uint32_t q = at.u / per, s = 0;
  int e = 0, row0 = 0, rows = 0;
  const uint8_t *x[kRows];  // in shared memory
  int my_row = -1;       // this lane's result: its row, channel and scales
  uint32_t my_n = 0;
  float xs = 0.0f, ws = 0.0f, ws_up = 0.0f;
  bool new_tile = true;
  int acc[4][kRows];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < kRows; ++r) acc[i][r] = 0;
  while (at.u < total) {
#pragma unroll
    for (int b = 0; b < kDepth; ++b) {
      if (at.u >= total) break;
      if (new_tile) {
        new_tile = false;
        e = expert_of((int)q);
        row0 = rt.off[e] + ((int)q - rt.tile[e]) * kRows;
        rows = min(kRows, rt.off[e + 1] - row0);
        const int r = SWIGLU ? lane >> 1 : lane >> 2;
        const int xr = lane < kRows ? fp8_x_row(a, row0 + min(lane, rows - 1)) : 0;
#pragma unroll
        for (int j = 0; j < kRows; ++j)  // a bad one (flagged) reads row 0
          x[j] = xsm + (size_t)max(0, __shfl_sync(0xffffffffu, xr, j)) * a.K;
        my_row = r < rows ? row0 + r : -1;
        const int xl = __shfl_sync(0xffffffffu, xr, r & (kRows - 1));
        xs = my_row >= 0 ? a.xs[max(0, xl)] : 0.0f;
      }
      if (s == 0) {  // the unit's scales, on the way until its end
        my_n = (at.u - q * per) * (SWIGLU ? 2 : 4) + (SWIGLU ? lane & 1 : lane & 3);
        const bool on = my_row >= 0 && my_n < a.N;
        ws = on ? a.wsc[0][(size_t)e * a.N + my_n] : 0.0f;
        if (SWIGLU) ws_up = on ? a.wsc[1][(size_t)e * a.N + my_n] : 0.0f;
      }
      const uint32_t k = min(s * 512 + lane * 16, a.K - 16);  // past K the weights are zeros
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r >= rows) break;  // the warp alike
        const uint4 xv = *(const uint4 *)(x[r] + k);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][r] = dot16(buf[b][i], xv, acc[i][r]);
      }
      load(buf[b]);
      if (++s < steps) continue;
      // ---- the unit is done
      s = 0;
      int mine = 0, mine_up = 0;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r >= rows) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int v = __reduce_add_sync(0xffffffffu, acc[i][r]);
          acc[i][r] = 0;
          if (SWIGLU) {
            if (lane == r * 2 + (i & 1)) (i < 2 ? mine : mine_up) = v;
          } else {
            if (lane == r * 4 + i) mine = v;
          }
        }
      }
      if (my_row >= 0 && my_n < a.N) {
        float y = (float)mine * (xs * ws);
        if (SWIGLU) y = fp8_swiglu_value(y, (float)mine_up * (xs * ws_up));
        fp8_store(a, my_row, my_n, y);
      }
      at.next();
      if (at.u < total && at.u - q * per >= per) {
        q = at.u / per;
        new_tile = true;
      }
    }
  }
}

template <bool SWIGLU>
cudaError_t run_few(Fp8Args &a, cudaStream_t stream) {
  const int sms = fp8_ctas();
  const uint32_t n = SWIGLU ? 2 : 4;
  fp8_set_tiles(a, (a.N + n - 1) / n, sms);
  auto kern = k_int8_few<SWIGLU>;
  const size_t smem = (size_t)a.n_x * a.K + fp8_tiles_smem(a.E);
  static std::atomic<bool> done[kMaxDevices];
  const cudaError_t e = allow_smem(kern, done);
  if (e != cudaSuccess) return e;
  return launch_k(kern, sms, kThreads, smem, stream, true, a);
}

}  // namespace

cudaError_t launch_int8_few(Fp8Args &a, bool swiglu, cudaStream_t stream) {
  return swiglu ? run_few<true>(a, stream) : run_few<false>(a, stream);
}

}  // namespace moe
