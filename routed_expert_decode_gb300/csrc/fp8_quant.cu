// fp8_quant.cu -- rows to e4m3 with a scale per 128 columns, and the weighted
// combine of the experts' output rows.  Both move each byte once and are bound
// by HBM for many rows, by the launch for few.
#include "fp8_common.cuh"

namespace moe {
namespace {

constexpr int kQuantWarps = 4;
constexpr int kQuantSteps = 2;                    // steps whose loads are in flight together
constexpr uint32_t kQuantSpan = 4 * kQuantSteps;  // blocks per warp: four a step

// scale = a / 448, q = rn_e4m3(x * (448 / a)), a = max(max|x|, 2^-100) over a block
// of 128 columns of a row.  Eight lanes hold a block, 16 values each, so the
// maximum is three shuffles and a lane's codes are one 16-byte store; a warp takes
// 8 consecutive blocks of one row with all its loads issued first (64 bytes a lane
// of a 16-bit type).  VEC: rows whose blocks are whole and 16-byte aligned.  8192 rows of
// 6144 bf16: 23.8 us, 6.4 TB/s; fp32 39.6 us, 6.4 TB/s.  Other widths load single elements
// and store single bytes, in every block: 6160 bf16 take 105 us.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kQuantWarps * 32)
    k_fp8_quantize(const void *x, size_t ld, uint32_t T, uint32_t d, uint32_t nb,
                   uint32_t spans, uint8_t *q, float *scale) {
  pdl_trigger();
  pdl_wait();
  using E = Elem<DT>;
  const int lane = threadIdx.x & 31, sub = lane >> 3, l8 = lane & 7;
  const uint64_t wi = (uint64_t)blockIdx.x * kQuantWarps + threadIdx.x / 32;
  if (wi >= (uint64_t)T * spans) return;
  const uint32_t t = (uint32_t)(wi / spans);
  const uint32_t b0 = (uint32_t)(wi - (uint64_t)t * spans) * kQuantSpan + sub;
  const typename E::T *row = (const typename E::T *)x + (size_t)t * ld;
  Raw8<DT> raw[kQuantSteps][2];
#pragma unroll
  for (int s = 0; s < kQuantSteps; ++s)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t c = (b0 + 4 * s) * kFp8Block + l8 * 16 + 8 * h;
      if (VEC) {
        if (b0 + 4 * s < nb) raw[s][h].load(row + c);
      } else {
        typename E::T *v = (typename E::T *)raw[s][h].v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = b0 + 4 * s < nb && c + i < d ? row[c + i] : E::from(0.0f);
      }
    }
#pragma unroll
  for (int s = 0; s < kQuantSteps; ++s) {
    const uint32_t b = b0 + 4 * s;
    const bool live = b < nb;
    float f[2][8], amax = 0.0f;
    if (live) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        raw[s][h].to(f[h]);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[h][i]));
      }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (!live) continue;
    float sc, inv;
    fp8_block_scale(amax, sc, inv);
    if (l8 == 0) scale[(size_t)t * nb + b] = sc;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float *v = f[i >> 1] + 4 * (i & 1);
      w[i] = e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    }
    const uint32_t c = b * kFp8Block + l8 * 16;
    uint8_t *dst = q + (size_t)t * d + c;
    if (VEC) {
      *(uint4 *)dst = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c + i < d) dst[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
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
                   (T == 1 || ld * dtype_size(DT) % 16 == 0) && ((uintptr_t)q & 15) == 0;
  return launch_k(vec ? k_fp8_quantize<DT, true> : k_fp8_quantize<DT, false>, grid,
                  kQuantWarps * 32, 0, stream, true, x, ld, T, d, nb, spans, (uint8_t *)q, scale);
}

constexpr int kCombThreads = 256;
constexpr int kCombBatch = 8;  // rows of o on the way together

// y[t] = shared[t] + sum_j w[t][j] o[pos[t][j]], fp32, slots in order.  8 columns a
// thread and step; up to 8 rows' loads (128 bytes of a 16-bit type a thread, 128 KB
// an SM) are issued before the first is used.  With enough tokens to fill the SMs a
// CTA walks a whole token (4096 tokens of 8 rows of 6144 columns: 79.7 us, 82.5 with
// its columns on three CTAs); with fewer a token's columns are spread over `parts`
// CTAs (one token: 2.6 us, 4.1 on one CTA).  Eight fp32 rows are all 64 registers of a
// thread: 276 bytes spill, and the same 4096 tokens in fp32 take 235 us, for bytes that a
// copy moves in 148.
template <int DT, int YT, bool VEC>
__global__ void __launch_bounds__(kCombThreads, 4)
    k_fp8_combine(const void *o, size_t ldo, uint32_t R, const float *w, const int32_t *pos,
                  uint32_t T, uint32_t k, uint32_t d, uint32_t parts, const void *shared, size_t lds,
                  void *y, size_t ldy) {
  pdl_trigger();
  pdl_wait();
  using E = Elem<DT>;
  using Y = Elem<YT>;
  const uint32_t items = T * parts;  // below 2^31, as the host checked
  for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
    const uint32_t t = item / parts;
    const uint32_t c0 = ((item - t * parts) * blockDim.x + threadIdx.x) * 8;
    const float *wt = w + (size_t)t * k;
    const int32_t *pt = pos + (size_t)t * k;
    for (uint32_t c = c0; c < d; c += parts * blockDim.x * 8) {
      auto load = [&](Raw8<DT> &raw, const void *base, size_t row, size_t ld) {
        const typename E::T *p = (const typename E::T *)base + row * ld + c;
        if (VEC) {
          raw.load(p);
        } else {
          typename E::T *v = (typename E::T *)raw.v;
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = c + i < d ? p[i] : E::from(0.0f);
        }
      };
      float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      Raw8<DT> first;
      if (shared) load(first, shared, t, lds);
      for (uint32_t j0 = 0; j0 < k; j0 += kCombBatch) {
        Raw8<DT> raw[kCombBatch];
        uint32_t pj[kCombBatch];
#pragma unroll
        for (int j = 0; j < kCombBatch; ++j) {
          pj[j] = j0 + j < k ? (uint32_t)pt[j0 + j] : R;
          if (pj[j] < R) load(raw[j], o, pj[j], ldo);
        }
        if (j0 == 0 && shared) first.to(acc);
#pragma unroll
        for (int j = 0; j < kCombBatch; ++j)
          if (pj[j] < R) {
            const float wj = wt[j0 + j];
            float f[8];
            raw[j].to(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = __fmaf_rn(wj, f[i], acc[i]);
          }
      }
      typename Y::T *dst = (typename Y::T *)y + (size_t)t * ldy + c;
      if (VEC) {
        store8<YT>(dst, acc);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < d) dst[i] = Y::from(acc[i]);
      }
    }
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
  const uint32_t need = (a.d + 255) / 256 * 32;  // threads for 8 columns each
  const uint32_t threads = need < kCombThreads ? need : kCombThreads;
  // as many at a time as the SMs hold
  const uint64_t most = (uint64_t)fp8_ctas() * (2048 / threads < 32 ? 2048 / threads : 32);
  const uint32_t parts = a.T < most ? (need + threads - 1) / threads : 1;
  const uint64_t items = (uint64_t)a.T * parts;
  const unsigned grid = (unsigned)(items < most ? items : most);
  auto ok = [](const void *p, size_t ld, size_t es) {
    return ((uintptr_t)p & 15) == 0 && ld * es % 16 == 0;
  };
  const bool vec = a.d % 8 == 0 && ok(a.o, a.ldo, dtype_size(DT)) &&
                   (!a.shared || ok(a.shared, a.lds, dtype_size(DT))) &&
                   ok(a.y, a.ldy, dtype_size(YT));
  return launch_k(vec ? k_fp8_combine<DT, YT, true> : k_fp8_combine<DT, YT, false>, grid,
                  threads, 0, a.stream, true, a.o, a.ldo, a.R, a.w, a.pos, a.T, a.k, a.d,
                  parts, a.shared, a.lds, a.y, a.ldy);
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
