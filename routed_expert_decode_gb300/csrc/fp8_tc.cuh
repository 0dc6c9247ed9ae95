// fp8_tc.cuh -- the tensor-core product (fp8_tc.cu), as fp8_gemm.cu calls it
#pragma once

#include "fp8_tiles.cuh"

namespace moe {

// operands that tensor copies can take: 16-byte aligned planes and rows
bool fp8_tc_ok(const Fp8Args &a);
// workspace bytes of its split tiles
size_t fp8_tc_ws(uint32_t rows);
// experts with many rows (fp8_tc.cu), and with few (fp8_tc_few.cu)
cudaError_t launch_fp8_tc(Fp8Args &a, bool swiglu, cudaStream_t stream);
cudaError_t launch_fp8_few(Fp8Args &a, bool swiglu, cudaStream_t stream);
// up to this many rows an expert, on average, the call is one of few rows
constexpr uint64_t kFp8FewRows = 64;

}  // namespace moe
