// fp8_common.cuh -- types and helpers shared by the block-scaled fp8 operators
// (moe_fp8.h): element loads and stores by type, e4m3 conversion, launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "fp8_host.h"
#include "moe_fp8.h"
#include "moe_internal.cuh"

namespace moe {

constexpr int kFp8Block = 128;              // weights: 128 x 128, activations: 1 x 128
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxMin = 0x1p-100f;       // smallest block maximum a scale is made from

__host__ __device__ constexpr uint32_t fp8_blocks(uint32_t n) {
  return n / kFp8Block + (n % kFp8Block != 0);
}

// words of the workspace's counter area (moe.h) used by these operators, clear
// of the layer's: zero between calls
constexpr uint32_t kFp8TileSync = 2080;      // [kFp8MaxCtas * 4]: parts of a split tile done
constexpr uint32_t kFp8MaxCtas = 256;
static_assert(kQueueTcDown + 2 <= kFp8TileSync &&
                  kFp8TileSync + kFp8MaxCtas * 4 <= MOE_SYNC_BYTES / 4 - 2,
              "counters overlap the layer's");

__host__ __device__ constexpr size_t dtype_size(int dt) { return dt == MOE_DT_F32 ? 4 : 2; }

template <int DT>
struct Elem;
template <>
struct Elem<MOE_DT_F32> {
  using T = float;
  static __device__ __forceinline__ float to(float v) { return v; }
  static __device__ __forceinline__ float from(float v) { return v; }
};
template <>
struct Elem<MOE_DT_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float to(T v) { return __bfloat162float(v); }
  static __device__ __forceinline__ T from(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<MOE_DT_F16> {
  using T = __half;
  static __device__ __forceinline__ float to(T v) { return __half2float(v); }
  static __device__ __forceinline__ T from(float v) { return __float2half_rn(v); }
};

// two values of a 16-bit type in one word, as floats, and back
template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if (DT == MOE_DT_BF16) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&v));
  return __half22float2(*reinterpret_cast<__half2 *>(&v));
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (DT == MOE_DT_BF16) {
    __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&r);
  }
  __half2 r = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t *>(&r);
}

// v / d with inv = floor((2^32 - 1) / d): the product's high word is at most one short
__device__ __forceinline__ uint32_t quotient(uint32_t v, uint32_t d, uint32_t inv) {
  const uint32_t q = __umulhi(v, inv);
  return v - q * d >= d ? q + 1 : q;
}

// 16 bytes, read once (no L1 allocation).  Volatile, and not a read-only load:
// a load of what the stream's previous kernel wrote must stay behind pdl_wait
__device__ __forceinline__ uint4 ld_once16(const void *p) {
  uint4 w;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "l"(p));
  return w;
}

// eight consecutive elements from a 16-byte (32-byte for fp32: two 16-byte
// loads) aligned place, as floats
template <int DT>
struct Raw8 {
  uint4 v[DT == MOE_DT_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void *p) {
#pragma unroll
    for (int i = 0; i < (DT == MOE_DT_F32 ? 2 : 1); ++i) v[i] = ld_once16((const uint4 *)p + i);
  }
  __device__ __forceinline__ void to(float (&f)[8]) const {
    if (DT == MOE_DT_F32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 w = v[DT == MOE_DT_F32 ? i : 0];
        f[4 * i] = __uint_as_float(w.x);
        f[4 * i + 1] = __uint_as_float(w.y);
        f[4 * i + 2] = __uint_as_float(w.z);
        f[4 * i + 3] = __uint_as_float(w.w);
      }
    } else {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t = unpack2<DT>(w[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
      }
    }
  }
};

template <int DT>
__device__ __forceinline__ void store8(void *p, const float (&f)[8]) {
  if (DT == MOE_DT_F32) {
    ((float4 *)p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    ((float4 *)p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *(uint4 *)p = make_uint4(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]), pack2<DT>(f[4], f[5]),
                             pack2<DT>(f[6], f[7]));
  }
}

// four floats -> four e4m3 bytes: nearest, ties to even, saturating at 448; NaN
// stays NaN
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ uint8_t e4m3x1(float a) {
  return (uint8_t)__nv_cvt_float_to_fp8(a, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float e4m3_to_float(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3)));
}

// a block's scale and the factor its values are multiplied by before rounding,
// from the largest |x| (one IEEE division each; NaN values do not enter amax)
__device__ __forceinline__ void fp8_block_scale(float amax, float &scale, float &inv) {
  const float a = fmaxf(amax, kAmaxMin);
  scale = __fdiv_rn(a, kE4m3Max);
  inv = __fdiv_rn(kE4m3Max, a);
}

// ---------------------------------------------------------------- launchers
// CTAs of a kernel that runs one per SM (a device's SM count is looked up once)
inline int fp8_ctas() {
  static std::atomic<int> known[kMaxDevices];
  const int dev = device_here();
  if (dev < 0) return kSmCount;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
      return kSmCount;
    n = n < (int)kFp8MaxCtas ? n : (int)kFp8MaxCtas;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}
cudaError_t launch_fp8_quantize(const void *x, int dt, size_t ld, uint32_t T, uint32_t d, void *q,
                                float *scale, cudaStream_t stream);
cudaError_t launch_fp8_combine(const void *o, int dt, size_t ldo, uint32_t R, const float *w,
                               const int32_t *pos, uint32_t T, uint32_t k, uint32_t d,
                               const void *shared, size_t lds, void *y, int ydt, size_t ldy,
                               cudaStream_t stream);
size_t group_route_ws(const moe_router &r);
cudaError_t launch_group_route(const moe_router &r, const void *logits, int dt, size_t ld,
                               const float *bias, uint32_t T, int32_t *idx, float *w,
                               int32_t *off, int32_t *perm, int32_t *pos, void *ws,
                               cudaStream_t stream);

// one product call; swiglu: two matrices and quantised outputs
struct Fp8Call {
  bool swiglu;
  moe_fp8_mat w[2];
  uint32_t E, N, K;
  moe_fp8_rows x;
  void *out;  // product output, or the h codes
  int odt;
  size_t ld;
  float *hs;
  uint8_t *ws;
  cudaStream_t stream;
};
size_t fp8_gemm_ws(uint32_t rows);
cudaError_t launch_fp8_gemm(const Fp8Call &c);

}  // namespace moe
