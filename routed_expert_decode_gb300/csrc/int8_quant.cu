// int8_quant.cu -- rows to int8 codes with one scale a row.  Moves each byte once and is
// bound by HBM for many rows, by the launch for few.
#include "int8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kSteps = 4;  // groups of 8 elements a thread keeps: rows of up to 32 a thread

// A team of 32 to 256 threads takes a row: all of it into registers (rows of more than
// 8192 columns go past twice), the maximum of |x| over the team, the codes.  |x| as its
// bit pattern is ordered with infinities above the numbers and NaN above those, so one
// integer maximum also tells a row that has either.  VEC: rows in 16-byte steps.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
    k_int8_quantize(const void *x, size_t ld, uint32_t T, uint32_t d, uint32_t team, uint8_t *q,
                    float *scale) {
  pdl_trigger();
  pdl_wait();
  using E = Elem<DT>;
  __shared__ uint32_t red[kThreads / 32];
  const uint32_t tid = threadIdx.x, m = tid / team, l = tid - m * team;
  const uint32_t t = blockIdx.x * (kThreads / team) + m;
  const bool on = t < T;
  const typename E::T *row = (const typename E::T *)x + (size_t)(on ? t : 0) * ld;
  const uint32_t span = team * 8;  // columns of a step
  Raw8<DT> raw[kSteps];
  auto load = [&](Raw8<DT> &r, uint32_t c) {
    if (VEC) {
      if (on && c < d) {
        r.load(row + c);
      } else {
#pragma unroll
        for (int i = 0; i < (DT == MOE_DT_F32 ? 2 : 1); ++i) r.v[i] = make_uint4(0, 0, 0, 0);
      }
    } else {
      typename E::T *v = (typename E::T *)r.v;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = on && c + i < d ? row[c + i] : E::from(0.0f);
    }
  };
  auto largest = [&](const Raw8<DT> &r, uint32_t a) {
    float f[8];
    r.to(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(fabsf(f[i])));
    return a;
  };
  uint32_t amax = 0;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) load(raw[s], l * 8 + s * span);
#pragma unroll
  for (int s = 0; s < kSteps; ++s) amax = largest(raw[s], amax);
  for (uint64_t c = (uint64_t)l * 8 + (uint64_t)kSteps * span; c < d; c += span) {
    Raw8<DT> r;
    load(r, (uint32_t)c);
    amax = largest(r, amax);
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  if (team > 32) {
    if ((tid & 31) == 0) red[tid / 32] = amax;
    __syncthreads();
    for (uint32_t w = m * team / 32; w < (m + 1) * team / 32; ++w) amax = max(amax, red[w]);
  }
  if (!on) return;
  const bool finite = amax < 0x7f800000u;
  const float a = fmaxf(__uint_as_float(amax), kAmaxMin);
  const float inv = finite ? __fdiv_rn(127.0f, a) : 0.0f;
  if (l == 0) scale[t] = finite ? __fdiv_rn(a, 127.0f) : __uint_as_float(0x7fffffffu);
  uint8_t *dst = q + (size_t)t * d;
  auto store = [&](const Raw8<DT> &r, uint32_t c) {
    float f[8];
    r.to(f);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int v = finite ? __float2int_rn(f[i] * inv) : 0;
      w[i / 4] |= (uint32_t)(v & 255) << (8 * (i % 4));
    }
    if (VEC) {
      if (c < d) *(uint2 *)(dst + c) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < d) dst[c + i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
  };
#pragma unroll
  for (int s = 0; s < kSteps; ++s) store(raw[s], l * 8 + s * span);
  for (uint64_t c = (uint64_t)l * 8 + (uint64_t)kSteps * span; c < d; c += span) {
    Raw8<DT> r;
    load(r, (uint32_t)c);
    store(r, (uint32_t)c);
  }
}

template <int DT>
cudaError_t quantize_t(const void *x, size_t ld, uint32_t T, uint32_t d, void *q, float *scale,
                       cudaStream_t stream) {
  uint32_t team = 32;  // as few threads as keep a row in registers
  while (team < kThreads && team * 8 * kSteps < d) team *= 2;
  const uint32_t rows = kThreads / team;
  const bool vec = d % 8 == 0 && ((uintptr_t)x & 15) == 0 &&
                   (T == 1 || ld * dtype_size(DT) % 16 == 0) && ((uintptr_t)q & 7) == 0;
  return launch_k(vec ? k_int8_quantize<DT, true> : k_int8_quantize<DT, false>,
                  (T + rows - 1) / rows, kThreads, 0, stream, true, x, ld, T, d, team,
                  (uint8_t *)q, scale);
}

}  // namespace

cudaError_t launch_int8_quantize(const void *x, int dt, size_t ld, uint32_t T, uint32_t d, void *q,
                                 float *scale, cudaStream_t stream) {
  if (dt == MOE_DT_F32) return quantize_t<MOE_DT_F32>(x, ld, T, d, q, scale, stream);
  if (dt == MOE_DT_BF16) return quantize_t<MOE_DT_BF16>(x, ld, T, d, q, scale, stream);
  return quantize_t<MOE_DT_F16>(x, ld, T, d, q, scale, stream);
}

}  // namespace moe
