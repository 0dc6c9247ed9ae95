// int8.cuh -- launchers of the int8 operators (moe_int8.h)
#pragma once

#include "fp8_tiles.cuh"
#include "moe_int8.h"

namespace moe {

cudaError_t launch_int8_quantize(const void *x, int dt, size_t ld, uint32_t T, uint32_t d, void *q,
                                 float *scale, cudaStream_t stream);

// One product call; swiglu: two matrices.  The kernels take an Fp8Args, whose xs is one
// scale a row, wsc one a channel and nbk the blocks of 128 along K.
struct Int8Call {
  bool swiglu;
  moe_int8_mat w[2];
  uint32_t E, N, K;
  moe_int8_rows x;
  void *out;
  int odt;
  size_t ld;
  uint8_t *ws;
  cudaStream_t stream;
};
size_t int8_gemm_ws();
cudaError_t launch_int8_gemm(const Int8Call &c);
// the same of a few rows in all on CUDA cores (int8_few.cu), same conditions
cudaError_t launch_int8_few(Fp8Args &a, bool swiglu, cudaStream_t stream);
// the tensor-core products (int8_tc.cu): operands that tensor copies can take
bool int8_tc_ok(const Fp8Args &a);
size_t int8_tc_ws();
cudaError_t launch_int8_tc(Fp8Args &a, bool swiglu, cudaStream_t stream);

}  // namespace moe
