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
// 32 experts, 4096 x 2048 (us; the few-row kernel's tiles of up to 32 rows, for the down
// product also of up to 64, and the many-row kernel):
//   rows       16        32        48        64        96       128
//   gate/up  87  92    87  95    94  97   107  99   140 105   182 130
//   down    47 47 53  48 49 55  59 50 56  71 54 59  99 61 65  126 76 66
// The same number of rows for every expert; where a router spreads them, the down
// product's 32-row tiles are 1 to 5 % ahead up to 48 (28 rows 48.7 and 49.1, 32 47.1 and
// 49.3, 40 49.9 and 50.4, 48 48.9 and 51.2).
constexpr uint64_t kFp8FewSwiglu = 48;  // tiles of 32 rows up to here
constexpr uint64_t kFp8FewProduct32 = 24, kFp8FewProduct64 = 96;

}  // namespace moe
