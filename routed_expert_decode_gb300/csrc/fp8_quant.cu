// fp8_quant.cu -- rows to e4m3 with a scale per 128 columns, and the weighted
// combine of the experts' output rows.  Both move each byte once and are bound
// by HBM for many rows, by the launch for few.
#include "fp8_common.cuh"

namespace moe {
namespace {

constexpr int kQuantWarps = 8;
constexpr int kQuantSteps = 4;                    // loads in flight per lane
constexpr uint32_t kQuantSpan = 2 * kQuantSteps;  // blocks per warp: two half-warps a step

// scale = a / 448, q = rn_e4m3(x * (448 / a)), a = max(max|x|, 2^-100) over a block
// of 128 columns of a row.  Half a warp holds a block, 8 values a lane, so the
// maximum is four shuffles; a warp takes 8 consecutive blocks of one row with all
// its loads issued first (64 bytes a lane of a 16-bit type in flight: the 2048
// threads of an SM keep ~128 KB on the way, well over the ~45 KB that HBM's
// latency asks for).  VEC: rows whose blocks are whole and 16-byte aligned.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kQuantWarps * 32)
    k_fp8_quantize(const void *x, size_t ld, uint32_t T, uint32_t d, uint32_t nb,
                   uint32_t spans, uint8_t *q, float *scale) {
  pdl_trigger();
  pdl_wait();
  using E = Elem<DT>;
  const int lane = threadIdx.x & 31, half = lane >> 4, l16 = lane & 15;
  const uint64_t wi = (uint64_t)blockIdx.x * kQuantWarps + threadIdx.x / 32;
  if (wi >= (uint64_t)T * spans) return;
  const uint32_t t = (uint32_t)(wi / spans);
  const uint32_t b0 = (uint32_t)(wi - (uint64_t)t * spans) * kQuantSpan + half;
  const typename E::T *row = (const typename E::T *)x + (size_t)t * ld;
  float f[kQuantSteps][8];
  if (VEC) {
    Raw8<DT> raw[kQuantSteps];
#pragma unroll
    for (int s = 0; s < kQuantSteps; ++s)
      if (b0 + 2 * s < nb) raw[s].load(row + (size_t)(b0 + 2 * s) * kFp8Block + l16 * 8);
#pragma unroll
    for (int s = 0; s < kQuantSteps; ++s)
      if (b0 + 2 * s < nb) raw[s].to(f[s]);
  } else {
#pragma unroll
    for (int s = 0; s < kQuantSteps; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t c = (b0 + 2 * s) * kFp8Block + l16 * 8 + i;
        f[s][i] = b0 + 2 * s < nb && c < d ? E::to(row[c]) : 0.0f;
      }
  }
#pragma unroll
  for (int s = 0; s < kQuantSteps; ++s) {
    const uint32_t b = b0 + 2 * s;
    const bool live = b < nb;
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, live ? fabsf(f[s][i]) : 0.0f);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (!live) continue;
    float sc, inv;
    fp8_block_scale(amax, sc, inv);
    if (l16 == 0) scale[(size_t)t * nb + b] = sc;
    const uint32_t c = b * kFp8Block + l16 * 8;
    uint8_t *dst = q + (size_t)t * d + c;
    if (VEC) {
      uint2 v;
      v.x = e4m3x4(f[s][0] * inv, f[s][1] * inv, f[s][2] * inv, f[s][3] * inv);
      v.y = e4m3x4(f[s][4] * inv, f[s][5] * inv, f[s][6] * inv, f[s][7] * inv);
      *(uint2 *)dst = v;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < d) dst[i] = e4m3x1(f[s][i] * inv);
    }
  }
}

template <int DT>
cudaError_t quantize_t(const void *x, size_t ld, uint32_t T, uint32_t d, void *q, float *scale,
                       cudaStream_t stream) {
  const uint32_t nb = fp8_blocks(d);
  const uint32_t spans = (nb + kQuantSpan - 1) / kQuantSpan;
  const uint64_t warps = (uint64_t)T * spans;
  const unsigned grid = (unsigned)((warps + kQuantWarps - 1) / kQuantWarps);
  const bool vec = d % kFp8Block == 0 && ((uintptr_t)x & 15) == 0 &&
                   (T == 1 || ld * dtype_size(DT) % 16 == 0) && ((uintptr_t)q & 7) == 0;
  return launch_k(vec ? k_fp8_quantize<DT, true> : k_fp8_quantize<DT, false>, grid,
                  kQuantWarps * 32, 0, stream, true, x, ld, T, d, nb, spans, (uint8_t *)q, scale);
}

constexpr int kCombWarps = 8;
constexpr int kCombBatch = 8;  // rows of o loaded before any is used

// y[t] = shared[t] + sum_j w[t][j] o[pos[t][j]], fp32, slots in order.  A warp takes
// 256 columns of a token (8 a lane) and issues up to 8 rows' loads together.
template <int DT, int YT, bool VEC>
__global__ void __launch_bounds__(kCombWarps * 32)
    k_fp8_combine(const void *o, size_t ldo, uint32_t R, const float *w,
                  const int32_t *pos, uint32_t T, uint32_t k, uint32_t d,
                  uint32_t segs, const void *shared, size_t lds,
                  void *y, size_t ldy) {
  pdl_trigger();
  pdl_wait();
  using E = Elem<DT>;
  using Y = Elem<YT>;
  const int lane = threadIdx.x & 31;
  const uint64_t wi = (uint64_t)blockIdx.x * kCombWarps + threadIdx.x / 32;
  if (wi >= (uint64_t)T * segs) return;
  const uint32_t t = (uint32_t)(wi / segs);
  const uint32_t c = (uint32_t)(wi - (uint64_t)t * segs) * 256 + lane * 8;
  // lane j holds slot j's weight and row
  float wl = 0.0f;
  int pl = -1;
  if ((uint32_t)lane < k) {
    wl = w[(size_t)t * k + lane];
    pl = pos[(size_t)t * k + lane];
    if ((uint32_t)pl >= R) pl = -1;
  }
  auto load = [&](const void *base, size_t row, size_t ld, float (&f)[8]) {
    const typename E::T *p = (const typename E::T *)base + row * ld + c;
    if (VEC) {
      Raw8<DT> raw;
      raw.load(p);
      raw.to(f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = c + i < d ? E::to(p[i]) : 0.0f;
    }
  };
  float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  const bool live = c < d;
  if (shared && live) load(shared, t, lds, acc);
  for (uint32_t j0 = 0; j0 < k; j0 += kCombBatch) {
    float f[kCombBatch][8], wj[kCombBatch];
    int pj[kCombBatch];
#pragma unroll
    for (int j = 0; j < kCombBatch; ++j) {
      const int src = min(j0 + j, 31u);
      wj[j] = __shfl_sync(0xffffffffu, wl, src);
      pj[j] = __shfl_sync(0xffffffffu, pl, src);
      if (j0 + j >= k) pj[j] = -1;
      if (pj[j] >= 0 && live) load(o, pj[j], ldo, f[j]);
    }
#pragma unroll
    for (int j = 0; j < kCombBatch; ++j)
      if (pj[j] >= 0 && live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __fmaf_rn(wj[j], f[j][i], acc[i]);
      }
  }
  if (!live) return;
  typename Y::T *dst = (typename Y::T *)y + (size_t)t * ldy + c;
  if (VEC) {
    store8<YT>(dst, acc);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < d) dst[i] = Y::from(acc[i]);
  }
}

struct CombineArgs {
  const void *o;
  size_t ldo;
  uint32_t R;
  const float *w;
  const int32_t *pos;
  uint32_t T, k, d;
  const void *shared;
  size_t lds;
  void *y;
  size_t ldy;
  cudaStream_t stream;
};

template <int DT, int YT>
cudaError_t combine_t(const CombineArgs &a) {
  const uint32_t segs = (a.d + 255) / 256;
  const uint64_t warps = (uint64_t)a.T * segs;
  const unsigned grid = (unsigned)((warps + kCombWarps - 1) / kCombWarps);
  auto ok = [](const void *p, size_t ld, size_t es) {
    return ((uintptr_t)p & 15) == 0 && ld * es % 16 == 0;
  };
  const bool vec = a.d % 8 == 0 && ok(a.o, a.ldo, dtype_size(DT)) &&
                   (!a.shared || ok(a.shared, a.lds, dtype_size(DT))) &&
                   ok(a.y, a.ldy, dtype_size(YT));
  return launch_k(vec ? k_fp8_combine<DT, YT, true> : k_fp8_combine<DT, YT, false>, grid,
                  kCombWarps * 32, 0, a.stream, true, a.o, a.ldo, a.R, a.w, a.pos, a.T, a.k, a.d,
                  segs, a.shared, a.lds, a.y, a.ldy);
}

template <int DT>
cudaError_t combine_from(int ydt, const CombineArgs &a) {
  if (ydt == MOE_DT_F32) return combine_t<DT, MOE_DT_F32>(a);
  if (ydt == MOE_DT_BF16) return combine_t<DT, MOE_DT_BF16>(a);
  return combine_t<DT, MOE_DT_F16>(a);
}

}  // namespace

cudaError_t launch_fp8_quantize(const void *x, int dt, size_t ld, uint32_t T, uint32_t d, void *q,
                                float *scale, cudaStream_t stream) {
  if (dt == MOE_DT_F32) return quantize_t<MOE_DT_F32>(x, ld, T, d, q, scale, stream);
  if (dt == MOE_DT_BF16) return quantize_t<MOE_DT_BF16>(x, ld, T, d, q, scale, stream);
  return quantize_t<MOE_DT_F16>(x, ld, T, d, q, scale, stream);
}

cudaError_t launch_fp8_combine(const void *o, int dt, size_t ldo, uint32_t R, const float *w,
                               const int32_t *pos, uint32_t T, uint32_t k, uint32_t d,
                               const void *shared, size_t lds, void *y, int ydt, size_t ldy,
                               cudaStream_t stream) {
  const CombineArgs a{o, ldo, R, w, pos, T, k, d, shared, lds, y, ldy, stream};
  if (dt == MOE_DT_F32) return combine_from<MOE_DT_F32>(ydt, a);
  if (dt == MOE_DT_BF16) return combine_from<MOE_DT_BF16>(ydt, a);
  return combine_from<MOE_DT_F16>(ydt, a);
}

}  // namespace moe
