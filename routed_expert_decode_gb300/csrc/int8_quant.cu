// int8_quant.cu -- rows to int8 codes with one scale a row.  Moves each byte once and is
// bound by HBM for many rows, by the launch for few.
#include "int8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// A team of 32 to 256 threads takes a row: all of it into registers (rows of more than
// 12288 columns go past twice), the maximum of |x| over the team, the codes.  |x| as its
// bit pattern is ordered with infinities above the numbers and NaN above those, so one
// integer maximum also tells a row that has either.  VEC: rows in 16-byte steps.  8192 rows of
// 6144: bf16 29 us, 5.2 TB/s, fp32 38, 6.6.
template <int DT, bool VEC, int kSteps>
__global__ void __launch_bounds__(kThreads, kSteps == 4 ? 4 : 3)
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
  auto largest = [&](const Raw8<DT> &r, float a) {  // a NaN stays
    float f[8];
    r.to(f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(fabsf(f[i])));
    return a;
  };
  float most = 0.0f;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) load(raw[s], l * 8 + s * span);
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
    if (l * 8 + s * span < d) most = largest(raw[s], most);
  for (uint64_t c = (uint64_t)l * 8 + (uint64_t)kSteps * span; c < d; c += span) {
    Raw8<DT> r;
    load(r, (uint32_t)c);
    most = largest(r, most);
  }
  uint32_t amax = __reduce_max_sync(0xffffffffu, __float_as_uint(most) & 0x7fffffffu);
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
    // x inv + 1.5 2^23: the sum's last bits are the rounded product in two's complement (ties
    // to even; the product is rounded to fp32 first, so the two are not one operation)
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = __float_as_uint(__fadd_rn(__fmul_rn(f[i], inv), 12582912.0f));
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = finite ? __byte_perm(__byte_perm(v[4 * i], v[4 * i + 1], 0x0040),
                                  __byte_perm(v[4 * i + 2], v[4 * i + 3], 0x0040), 0x5410)
                    : 0;
    if (VEC) {
      if (c < d) *(uint2 *)(dst + c) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < d) dst[c + i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
  };
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
    if (l * 8 + s * span < d) store(raw[s], l * 8 + s * span);
  for (uint64_t c = (uint64_t)l * 8 + (uint64_t)kSteps * span; c < d; c += span) {
    Raw8<DT> r;
    load(r, (uint32_t)c);
    store(r, (uint32_t)c);
  }
}

template <int DT>
cudaError_t quantize_t(const void *x, size_t ld, uint32_t T, uint32_t d, void *q, float *scale,
                       cudaStream_t stream) {
  // four steps a thread, or six where only those hold the row, or (16-bit types) hold it with
  // less to spare: 8192 rows of 6144 bf16 29 us on 128 threads, 34 on 256
  auto fit = [&](uint32_t steps) {
    uint32_t team = 32;
    while (team < kThreads && team * 8 * steps < d) team *= 2;
    return team;
  };
  const uint32_t four = fit(4), six = fit(6);
  const bool use6 = six * 48 >= d && (four * 32 < d || (DT != MOE_DT_F32 && six * 6 < four * 4));
  const uint32_t team = use6 ? six : four, rows = kThreads / team;
  const bool vec = d % 8 == 0 && ((uintptr_t)x & 15) == 0 &&
                   (T == 1 || ld * dtype_size(DT) % 16 == 0) && ((uintptr_t)q & 7) == 0;
  auto run = [&](auto kern) {
    return launch_k(kern, (T + rows - 1) / rows, kThreads, 0, stream, true, x, ld, T, d, team,
                    (uint8_t *)q, scale);
  };
  if (use6) return vec ? run(k_int8_quantize<DT, true, 6>) : run(k_int8_quantize<DT, false, 6>);
  return vec ? run(k_int8_quantize<DT, true, 4>) : run(k_int8_quantize<DT, false, 4>);
}

}  // namespace

cudaError_t launch_int8_quantize(const void *x, int dt, size_t ld, uint32_t T, uint32_t d, void *q,
                                 float *scale, cudaStream_t stream) {
  if (dt == MOE_DT_F32) return quantize_t<MOE_DT_F32>(x, ld, T, d, q, scale, stream);
  if (dt == MOE_DT_BF16) return quantize_t<MOE_DT_BF16>(x, ld, T, d, q, scale, stream);
  return quantize_t<MOE_DT_F16>(x, ld, T, d, q, scale, stream);
}

}  // namespace moe
