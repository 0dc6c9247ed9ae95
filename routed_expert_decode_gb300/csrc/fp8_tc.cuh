// fp8_tc.cuh -- the tensor-core product (fp8_tc.cu), as fp8_gemm.cu calls it
#pragma once

#include "fp8_tiles.cuh"

namespace moe {

// operands that tensor copies can take: 16-byte aligned planes and rows
bool fp8_tc_ok(const Fp8Args &a);
// workspace bytes of its split tiles
size_t fp8_tc_ws(uint32_t rows);
cudaError_t launch_fp8_tc(Fp8Args &a, bool swiglu, cudaStream_t stream);

}  // namespace moe
