// fp8_tc.cuh -- the tensor-core product (fp8_tc.cu), as fp8_gemm.cu calls it
#pragma once

#include "fp8_tiles.cuh"

namespace moe {

// operands that tensor copies can take: 16-byte aligned planes and rows
bool fp8_tc_ok(const Fp8Args &a);
// workspace bytes of one share of a split tile, and of all: two a CTA
size_t fp8_part_bytes(uint32_t rows);
size_t fp8_tc_ws(uint32_t rows);
// experts with many rows (fp8_tc.cu), and with few (fp8_tc_few.cu)
cudaError_t launch_fp8_tc(Fp8Args &a, bool swiglu, cudaStream_t stream);
cudaError_t launch_fp8_few(Fp8Args &a, bool swiglu, cudaStream_t stream);
// The call's rows an expert, on average, choose the kernel and the few-row one's tile.
// 32 experts, 4096 x 2048 (us; tiles of up to 32 and 64 rows of the few-row kernel, the
// many-row kernel):
//   rows         16            32            48            64            96
//   gate/up   90  94 100    88 100 104   100 103 106   120 116 109   163 145 116
//   down      48  48  61    59  51  63    80  52  64    96  59  67   134  71  72
constexpr uint64_t kFp8FewSwiglu = 48;  // tiles of 32 rows up to here
constexpr uint64_t kFp8FewProduct32 = 24, kFp8FewProduct64 = 96;

}  // namespace moe
