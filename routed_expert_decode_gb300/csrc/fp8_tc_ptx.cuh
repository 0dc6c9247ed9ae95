// fp8_tc_ptx.cuh -- what the two tensor-core product kernels share: PTX helpers, a
// segment of work (and the few-row kernel's split), the tensor maps.
#pragma once

#include <cuda.h>

#include "fp8_tc.cuh"

namespace moe {

constexpr int kMaxStages = 12;
constexpr uint32_t kWBytes = 128 * 128;  // one weight box: 128 rows of one K block
constexpr int kMinShare = 4;             // K blocks a CTA takes of a split round, at least
constexpr long long kWaitCycles = 4000000000ll;  // ~2 s
constexpr int kSpin = 1 << 26;
constexpr int kHintNs = 20000;  // try_wait suspend-time hint: waiting warps sleep, not spin

// ---------------------------------------------------------------- PTX helpers
__device__ __forceinline__ uint32_t s32(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void bar_init(uint64_t *b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(s32(b)), "r"(n));
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(s32(b)) : "memory");
}
// the same by one lane of a converged warp, without a branch.  What each lane has
// waited for happens before what the barrier's waiters do next: a tcgen05.commit's
// arrival, which an asynchronous operation makes, does not carry that on.
__device__ __forceinline__ void bar_arrive_elect(uint64_t *b) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(s32(b))
      : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(s32(b)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t *b, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(s32(b)), "r"(parity), "n"(kHintNs)
      : "memory");
  return done != 0;
}
// the same without suspending the thread
__device__ __forceinline__ bool bar_test(uint64_t *b, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(s32(b)), "r"(parity)
      : "memory");
  return done != 0;
}
// What a wait that runs out does: it flags the call and sets the CTA's abort flag,
// after which every wait returns at once.  The work goes on to the end of the
// segment on whatever the buffers hold, so that a warp's lanes never part in front
// of a warp-wide instruction, and the roles' loops end there.
struct Guard {
  uint32_t *err;
  volatile int *abort_flag;
  // by a whole warp
  __device__ __forceinline__ bool aborted() const {
    return __any_sync(0xffffffffu, *abort_flag != 0);
  }
};
// bounded by a clock budget and a count; false: it ran out
__device__ __forceinline__ bool bar_wait_for(uint64_t *b, uint32_t parity) {
  const long long t0 = clock64();
  for (int i = 0; i < kSpin; ++i) {
    if (bar_try(b, parity)) return true;
    if (clock64() - t0 > kWaitCycles) return false;
  }
  return false;
}
__device__ __forceinline__ void bar_wait(uint64_t *b, uint32_t parity, const Guard &g) {
  if (bar_try(b, parity) || *g.abort_flag) return;
  const long long t0 = clock64();
  for (int i = 0; i < kSpin && !*g.abort_flag; ++i) {
    if (bar_try(b, parity)) return;
    if (clock64() - t0 > kWaitCycles) break;
  }
  if (!*g.abort_flag) atomicOr(g.err, kErrTimeout);
  *g.abort_flag = 1;
}
__device__ __forceinline__ void tma_w(void *dst, const CUtensorMap *map, int k, int n, int e,
                                      uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(s32(dst)),
      "l"(map), "r"(k), "r"(n), "r"(e), "r"(s32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_x(void *dst, const CUtensorMap *map, int k, int row,
                                      uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(s32(dst)),
      "l"(map), "r"(k), "r"(row), "r"(s32(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// 16 bytes global -> shared past L1, zeros beyond `bytes` of them; nothing unless go
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes, bool go) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %3, 0;\n"
      " @p cp.async.cg.shared.global [%0], [%1], 16, %2;\n}\n" ::"r"(dst),
      "l"(src), "r"(bytes), "r"((int)go)
      : "memory");
}
// 4 bytes global -> shared
__device__ __forceinline__ void cp4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// this thread arrives on b once its copies so far have landed
__device__ __forceinline__ void cp_arrive(uint64_t *b) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(s32(b)) : "memory");
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// The products of one block of 128 along K, D = A B^T from zero: four MMAs of K = 32,
// 32 bytes apart along the operands' rows (2 in the descriptors' units).  Called by
// a whole converged warp with uniform operands; one lane issues.
__device__ __forceinline__ void tc_mma_block(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred e, f, t;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n"
      " add.s64 a1, %1, 2;\n add.s64 a2, %1, 4;\n add.s64 a3, %1, 6;\n"
      " add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"
      " setp.ne.b32 f, 0, 0;\n setp.eq.b32 t, 0, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, f;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, t;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc)
      : "memory");
}
// arrive on b when the MMAs so far are done
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          s32(bar))
      : "memory");
}
// 32 consecutive fp32 columns of this warp's 32 TMEM lanes, no wait
__device__ __forceinline__ void tc_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// waits for the warp's loads; the registers of v pass through it so that no use of
// them can move above the wait
__device__ __forceinline__ void tc_wait_ld32(float (&v)[32]) {
#define R4(i) "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3])
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : R4(0), R4(4), R4(8), R4(12), R4(16), R4(20), R4(24), R4(28)::"memory");
}
#undef R4
__device__ __forceinline__ void st_global32(void *p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// shared-memory matrix descriptor: K-major operand, 128-byte swizzle (8-row groups
// of 1024 bytes), version 1
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// instruction descriptor: D f32, A and B e4m3, both K-major, N >> 3 at bit 17, M = 128
__device__ __forceinline__ uint32_t idesc_for(uint32_t n) {
  return (1u << 4) | ((n >> 3) << 17) | (8u << 24);
}

// a place in a ring of n stages: its index and the parity of its current use
struct Ring {
  uint32_t i = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++i == n) {
      i = 0;
      phase ^= 1;
    }
  }
};

// ---------------------------------------------------------------- work split
// K blocks kb0 .. kb1 - 1 of a tile
struct Seg {
  int tile, kb0, kb1;
};
// A CTA has in order: its share [pos, end) of the split tiles' K blocks, then whole
// tiles split, split + G, ...  Every role walks the same list.
struct Walk {
  int n_all, share, kbs, grid;  // tiles, K blocks per worker of the split tiles, per tile
  int pos, end, next;
  // the last, partial round is split if it has fewer than split_below tiles
  __device__ Walk(int n_all_, const Fp8Args &a, int worker, int workers, int split_below)
      : n_all(n_all_), kbs((int)a.nbk), grid(workers) {
    // 32 bits hold them: below 256 split tiles of at most 2^17 K blocks
    const int rest = n_all - grid * (int)quotient(n_all, grid, a.workers_inv);
    const int split = rest < split_below ? rest : 0;
    const int items = split * kbs;
    share = max((int)quotient(items + grid - 1, grid, a.workers_inv), min(kMinShare, kbs));
    pos = min(items, worker * share);
    end = min(items, pos + share);
    next = split + worker;
  }
  __device__ bool take(Seg &s) {
    if (pos < end) {
      s.tile = pos / kbs;
      s.kb0 = pos - s.tile * kbs;
      s.kb1 = min(kbs, s.kb0 + end - pos);
      pos += s.kb1 - s.kb0;
      return true;
    }
    if (next >= n_all) return false;
    s.tile = next;
    s.kb0 = 0;
    s.kb1 = kbs;
    next += grid;
    return true;
  }
  // workers that share split tile v
  __device__ int first_worker(int v) const { return v * kbs / share; }
  __device__ int last_worker(int v) const { return ((v + 1) * kbs - 1) / share; }
};

// ---------------------------------------------------------------- host
struct Fp8Maps {
  CUtensorMap x;     // [n_x][K] codes, box 128 x MT (rows in order)
  CUtensorMap w[2];  // [E][N][K] codes, box 128 x 128
};

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_fn() {
  static EncodeTiled fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeTiled)p;
  }();
  return fn;
}

// byte matrices [d2][d1][K], box 128 bytes of box_rows rows, 128-byte swizzle
inline bool byte_map(CUtensorMap *m, const void *base, uint64_t K, uint64_t d1, uint64_t d2, int dims,
              uint32_t box_rows) {
  const cuuint64_t size[3] = {K, d1, d2};
  const cuuint64_t stride[2] = {K, K * d1};
  const cuuint32_t box[3] = {128, box_rows, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, dims, const_cast<void *>(base), size, stride,
                     box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe
