// group_route.cu -- group-limited top-k routing and the stable permutation of
// the (token, slot) rows by expert, in one kernel.
//
// Selection, one warp per token.  The token's logits go to shared memory, where one
// rolled loop turns them into selection values c (the code runs from a cold
// instruction cache once per call: unrolled over a lane's experts it took 4.3 us a
// token, 2000 instructions).  Then lane l holds the NPER consecutive experts
// [l*NPER, (l+1)*NPER), so "lowest index" is "lowest lane, then lowest register"
// and a group of experts is a run of lanes: where the group size is NPER times a
// power of two, a group's best two c meet by shuffles inside the run; other
// sizes are scanned in shared memory.  Scores become order-preserving unsigned
// keys; a round of top-k is one redux.sync maximum, one ballot (the lowest lane
// that holds it wins) and a rescan of the winner's registers.
//
// Permutation.  A token picks an expert at most once, so the rank of row (t, j)
// among its expert's rows of a run of tokens is a population count: bit t of the
// expert's token mask is set, and the bits below t are the rows before it.  No
// order of atomics enters the result.  Each CTA owns a contiguous run of
// tokens, writes its count per expert, and after a grid-wide barrier adds up
// the counts of the CTAs before it and of the experts before each expert.  A
// call of a few rows counts them directly.
//
// What bounds it: the issue slots for many tokens (the logits are read once);
// for few tokens the chain load -> score -> k rounds in one CTA.
#include <float.h>

#include "fp8_common.cuh"

namespace moe {
namespace {

constexpr int kGrWarps = 32;
constexpr int kGrThreads = kGrWarps * 32;
constexpr uint32_t kGrMaskTokens = 128;  // tokens ranked at a time: 4 mask words per expert
constexpr uint32_t kGrMaskWords = kGrMaskTokens / 32;
constexpr uint32_t kGrSoloTokens = kGrWarps;  // up to one token a warp: one CTA, no barrier
constexpr uint32_t kGrFewRows = 64;  // up to here, rows are ranked by comparing them all
constexpr long long kGrWaitCycles = 4000000000ll;
constexpr int kGrSpinIters = 1 << 26;

struct GrArgs {
  moe_router r;
  const void *logits;
  int dt;
  size_t ld;
  const float *bias;
  uint32_t T, gsize, per_cta;  // experts per group, tokens per CTA
  int32_t *idx;
  float *w;
  int32_t *off, *perm, *pos;
  int32_t *hist;   // [grid][E]: rows of each CTA's tokens per expert
  uint32_t *sync;  // [2]
  uint32_t *err;
};

// order-preserving map of a float (never NaN) to an unsigned above 0; -0 as +0
__device__ __forceinline__ uint32_t order_key(float c) {
  const uint32_t b = __float_as_uint(c + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ float no_nan(float v) { return v == v ? v : -INFINITY; }

__device__ __forceinline__ float logit_value(float v) { return fminf(no_nan(v), FLT_MAX); }
__device__ __forceinline__ float load_logit(const void *p, int dt, size_t i) {
  float v;
  if (dt == MOE_DT_F32) v = ((const float *)p)[i];
  else if (dt == MOE_DT_BF16) v = __bfloat162float(((const __nv_bfloat16 *)p)[i]);
  else v = __half2float(((const __half *)p)[i]);
  return logit_value(v);
}
// a token's E logits to shared memory by its warp
template <int DT>
__device__ __forceinline__ void stage_logits(const void *p, size_t row, uint32_t E, int lane,
                                             float *sl) {
  const typename Elem<DT>::T *src = (const typename Elem<DT>::T *)p + row;
#pragma unroll 8
  for (uint32_t i = lane; i < E; i += 32) sl[i] = logit_value(Elem<DT>::to(src[i]));
}

// sigmoid and sqrt(softplus) with CUDA's expf and log1pf; -inf gives 0
__device__ __forceinline__ float sigmoid_of(float l) { return __frcp_rn(1.0f + expf(-l)); }
__device__ __forceinline__ float softplus_root_of(float l) {
  return __fsqrt_rn(fmaxf(l, 0.0f) + log1pf(expf(-fabsf(l))));
}
// e^(l - max) of a row: 0 at -inf, a row of nothing else included
__device__ __forceinline__ float softmax_term(float l, float m) {
  return l == -INFINITY ? 0.0f : expf(l - m);
}

// One token by one warp: its picks to idx/w and to s_pick (shared, [32]).
// sc: 32 * NPER floats of shared memory of the warp.
template <int NPER>
__device__ __forceinline__ void route_token(const GrArgs &a, uint32_t t, int lane, int32_t *s_pick,
                                            float *sc) {
  const uint32_t E = a.r.n_expert, k = a.r.top_k, G = a.r.n_group;
  const uint32_t e0 = (uint32_t)lane * NPER;
  const size_t row = (size_t)t * a.ld;
  const uint32_t fn = a.r.score;
  __syncwarp();
  if (a.dt == MOE_DT_F32) stage_logits<MOE_DT_F32>(a.logits, row, E, lane, sc);
  else if (a.dt == MOE_DT_BF16) stage_logits<MOE_DT_BF16>(a.logits, row, E, lane, sc);
  else stage_logits<MOE_DT_F16>(a.logits, row, E, lane, sc);
  // each lane's own entries so far: no warp barrier needed until the runs are read
  float m = -INFINITY, rsum = 0.0f;  // softmax: the row's maximum and 1 / sum
  if (fn == MOE_SCORE_SOFTMAX) {
#pragma unroll 1
    for (uint32_t i = lane; i < E; i += 32) m = fmaxf(m, sc[i]);
    m = key_value(__reduce_max_sync(0xffffffffu, order_key(m)));
    float sum = 0.0f;
#pragma unroll 1
    for (uint32_t i = lane; i < E; i += 32) sum += softmax_term(sc[i], m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    rsum = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
  }
  auto score = [&](float l) {
    return fn == MOE_SCORE_SIGMOID ? sigmoid_of(l)
           : fn == MOE_SCORE_SOFTMAX ? softmax_term(l, m) * rsum : softplus_root_of(l);
  };
  // selection values; by logit, they are what is staged
  if (fn != MOE_SCORE_SOFTMAX || a.bias || a.r.group_score != MOE_GROUP_MAX) {
#pragma unroll 1
    for (uint32_t i = lane; i < E; i += 32) {
      const float p = score(sc[i]);
      sc[i] = a.bias ? no_nan(p + a.bias[i]) : p;
    }
  }
  __syncwarp();
  uint32_t key[NPER];
  if (NPER % 4 == 0) {  // 16 bytes a load: free of bank conflicts
#pragma unroll
    for (int i = 0; i < NPER; i += 4) {
      const float4 v = *(const float4 *)(sc + e0 + i);
      key[i] = order_key(v.x);
      key[(i + 1) % NPER] = order_key(v.y);
      key[(i + 2) % NPER] = order_key(v.z);
      key[(i + 3) % NPER] = order_key(v.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPER; ++i) key[i] = order_key(sc[e0 + i]);
  }
#pragma unroll
  for (int i = 0; i < NPER; ++i) key[i] = e0 + i < E ? key[i] : 0u;
  // ---- groups: drop the experts of those that are not kept
  if (a.r.topk_group < G) {
    const uint32_t gs = a.gsize;
    const bool two = a.r.group_score == MOE_GROUP_TOP2_SUM && gs > 1;
    const uint32_t run = gs / NPER;
    float mine = -INFINITY;  // lane g: the score of group g
    if (gs % NPER == 0 && (run & (run - 1)) == 0) {
      uint32_t b1 = 0u, b2 = 0u;  // the two best keys
#pragma unroll
      for (int i = 0; i < NPER; ++i) {
        b2 = max(b2, min(b1, key[i]));
        b1 = max(b1, key[i]);
      }
#pragma unroll 1
      for (uint32_t o = 1; o < run; o <<= 1) {
        const uint32_t p1 = __shfl_xor_sync(0xffffffffu, b1, o);
        const uint32_t p2 = __shfl_xor_sync(0xffffffffu, b2, o);
        b2 = max(max(b2, p2), min(b1, p1));
        b1 = max(b1, p1);
      }
      const float s = two ? no_nan(key_value(b1) + key_value(b2)) : key_value(b1);
      mine = __shfl_sync(0xffffffffu, s, min((uint32_t)lane * run, 31u));
    } else if ((uint32_t)lane < G) {
      float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll 1
      for (uint32_t i = 0; i < gs; ++i) {
        const float v = sc[lane * gs + i];
        b2 = fmaxf(b2, fminf(b1, v));
        b1 = fmaxf(b1, v);
      }
      mine = two ? no_nan(b1 + b2) : b1;
    }
    __syncwarp();
    const uint32_t gk = (uint32_t)lane < G ? order_key(mine) : 0u;
    uint32_t before = 0;  // groups that go before this lane's
#pragma unroll 1
    for (uint32_t g = 0; g < G; ++g) {
      const uint32_t ok = __shfl_sync(0xffffffffu, gk, g);
      before += ok > gk || (ok == gk && g < (uint32_t)lane);
    }
    const uint32_t kept =
        __ballot_sync(0xffffffffu, (uint32_t)lane < G && before < a.r.topk_group);
    if (gs % NPER == 0) {  // a lane's experts are of one group
      if (!((kept >> (e0 / gs)) & 1u)) {
#pragma unroll
        for (int i = 0; i < NPER; ++i) key[i] = 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NPER; ++i)
        if (e0 + i < E && !((kept >> ((e0 + i) / gs)) & 1u)) key[i] = 0u;
    }
  }
  // ---- top k
  uint32_t best = 0u;
#pragma unroll
  for (int i = 0; i < NPER; ++i) best = max(best, key[i]);
  int mine = 0;  // lane j: the expert of slot j
#pragma unroll 1
  for (uint32_t j = 0; j < k; ++j) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const int win = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
    int at = 0;  // the winner's first register that holds it
    if (lane == win) {
#pragma unroll
      for (int i = NPER - 1; i >= 0; --i) at = key[i] == top ? i : at;
      best = 0u;
#pragma unroll
      for (int i = 0; i < NPER; ++i) {
        key[i] = i == at ? 0u : key[i];
        best = max(best, key[i]);
      }
    }
    const int e = win * NPER + __shfl_sync(0xffffffffu, at, win);
    if ((uint32_t)lane == j) mine = e;
  }
  // ---- weights: lane j evaluates its pick's p again from the logit
  const bool pick = (uint32_t)lane < k;
  const float p = pick ? score(load_logit(a.logits, a.dt, row + mine)) : 0.0f;
  float w = a.r.s * p;
  if (a.r.renorm) {
    float sum = p;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f;
  }
  if (pick) {
    a.idx[(size_t)t * k + lane] = mine;
    a.w[(size_t)t * k + lane] = w;
    s_pick[lane] = mine;
  }
}

// grid-wide barrier on sync[0] (CTAs in) and sync[1] (CTAs out; the last one
// zeroes both).  The launch is cooperative, so every CTA is resident; the wait
// is bounded all the same.  False: it gave up.
__device__ bool grid_barrier(uint32_t *sync, uint32_t n, uint32_t *err) {
  __shared__ int ok;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    ok = 1;
    atomicAdd(sync, 1u);
    const long long t0 = clock64();
    volatile uint32_t *in = sync;
    int i = 0;
    while (*in < n) {
      if (++i > kGrSpinIters || clock64() - t0 > kGrWaitCycles) {
        atomicOr(err, kErrTimeout);
        ok = 0;
        break;
      }
    }
    __threadfence();
    if (ok && atomicAdd(sync + 1, 1u) == n - 1) {
      atomicExch(sync, 0u);
      atomicExch(sync + 1, 0u);
    }
  }
  __syncthreads();
  return ok != 0;
}

template <int NPER>
__global__ void __launch_bounds__(kGrThreads, 1) k_group_route(const GrArgs a, const bool few) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ __align__(16) uint8_t gsm[];
  const uint32_t E = a.r.n_expert, k = a.r.top_k;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float *sc = (float *)gsm + warp * (32 * NPER);  // a warp's staged logits
  int32_t *s_pick = (int32_t *)gsm + blockDim.x * NPER;  // [kGrWarps][32]: latest picks
  uint32_t *mask = (uint32_t *)(s_pick + kGrWarps * 32);  // [E][kGrMaskWords]
  int32_t *cnt = (int32_t *)(mask + E * kGrMaskWords);    // [E]: rows, then next row per expert
  int32_t *scan = cnt + E;                        // [32]
  const bool solo = gridDim.x == 1;
  const uint32_t t0 = min(a.T, blockIdx.x * a.per_cta), t1 = min(a.T, t0 + a.per_cta);
  const uint32_t n_warps = blockDim.x / 32;

  if (few) {
    if ((uint32_t)warp < a.T) route_token<NPER>(a, warp, lane, s_pick + warp * 32, sc);
    __syncthreads();
    const uint32_t R = a.T * k;
    for (uint32_t e = tid; e <= E; e += blockDim.x) {
      int n = 0;
      for (uint32_t t = 0; t < a.T; ++t)
        for (uint32_t j = 0; j < k; ++j) n += s_pick[t * 32 + j] < (int)e;
      a.off[e] = n;
    }
    for (uint32_t r = tid; r < R; r += blockDim.x) {
      const uint32_t tr = r / k;
      const int e = s_pick[tr * 32 + r - tr * k];
      int rank = 0;
      for (uint32_t t = 0; t < a.T; ++t)
        for (uint32_t j = 0; j < k; ++j) {
          const int v = s_pick[t * 32 + j];
          rank += v < e || (v == e && t < tr);
        }
      a.perm[rank] = (int32_t)r;
      a.pos[r] = rank;
    }
    return;
  }
  for (uint32_t i = tid; i < E; i += kGrThreads) cnt[i] = 0;
  __syncthreads();
  for (uint32_t t = t0 + warp; t < t1; t += n_warps) {
    route_token<NPER>(a, t, lane, s_pick + warp * 32, sc);
    if ((uint32_t)lane < k) atomicAdd(&cnt[s_pick[warp * 32 + lane]], 1);
  }
  __syncthreads();

  // ---- rows of earlier CTAs and of all, per expert (thread e, e + 1024 > E never)
  int before = 0, total = 0;
  if (solo) {
    if ((uint32_t)tid < E) total = cnt[tid];
  } else {
    for (uint32_t e = tid; e < E; e += kGrThreads)
      __stcg(a.hist + (size_t)blockIdx.x * E + e, cnt[e]);
    if (!grid_barrier(a.sync, gridDim.x, a.err)) return;
    // kGrThreads / E threads an expert share the CTAs' rows
    int32_t *part = (int32_t *)mask;  // [2][E], free until the ranking
    for (uint32_t e = tid; e < 2 * E; e += kGrThreads) part[e] = 0;
    __syncthreads();
    const uint32_t lanes = max(1u, (uint32_t)kGrThreads / E);
    const uint32_t e = (uint32_t)tid % E, p = (uint32_t)tid / E;
    if (p < lanes) {
      int b = 0, s = 0;
#pragma unroll 8
      for (uint32_t q = p; q < gridDim.x; q += lanes) {
        const int v = __ldcg(a.hist + (size_t)q * E + e);
        s += v;
        if (q < blockIdx.x) b += v;
      }
      atomicAdd(&part[e], s);  // integer sums: any order gives the same
      atomicAdd(&part[E + e], b);
    }
    __syncthreads();
    if ((uint32_t)tid < E) {
      total = part[tid];
      before = part[E + tid];
    }
    __syncthreads();
  }
  // exclusive scan of the totals over the experts (thread e holds expert e)
  int incl = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int v = scan[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    scan[lane] = v;
  }
  __syncthreads();
  const int first = incl - total + (warp > 0 ? scan[warp - 1] : 0);
  if ((uint32_t)tid < E) {
    if (blockIdx.x == 0) {
      a.off[tid] = first;
      if ((uint32_t)tid == E - 1) a.off[E] = first + total;
    }
    cnt[tid] = first + before;  // this CTA's next row of expert tid
  }
  // ---- rank and place this CTA's rows, kGrMaskTokens tokens at a time
  for (uint32_t c0 = t0; c0 < t1; c0 += kGrMaskTokens) {
    const uint32_t n = min(kGrMaskTokens, t1 - c0) * k;
    __syncthreads();
    for (uint32_t i = tid; i < E * kGrMaskWords; i += kGrThreads) mask[i] = 0u;
    __syncthreads();
    for (uint32_t i = tid; i < n; i += kGrThreads) {
      const uint32_t tl = i / k;
      atomicOr(&mask[a.idx[(size_t)c0 * k + i] * kGrMaskWords + (tl >> 5)], 1u << (tl & 31));
    }
    __syncthreads();
    for (uint32_t i = tid; i < n; i += kGrThreads) {
      const uint32_t tl = i / k;
      const int e = a.idx[(size_t)c0 * k + i];
      int rank = cnt[e];
      for (uint32_t q = 0; q < (tl >> 5); ++q) rank += __popc(mask[e * kGrMaskWords + q]);
      rank += __popc(mask[e * kGrMaskWords + (tl >> 5)] & ((1u << (tl & 31)) - 1u));
      const size_t r = (size_t)c0 * k + i;
      a.perm[rank] = (int32_t)r;
      a.pos[r] = rank;
    }
    __syncthreads();
    if ((uint32_t)tid < E) {
      int add = 0;
#pragma unroll
      for (uint32_t q = 0; q < kGrMaskWords; ++q) add += __popc(mask[tid * kGrMaskWords + q]);
      cnt[tid] += add;
    }
  }
}

// tokens per CTA and CTAs of a call
void gr_split(uint32_t T, uint32_t sms, uint32_t *per, uint32_t *grid) {
  if (T <= kGrSoloTokens) {
    *per = kGrSoloTokens;
    *grid = 1;
    return;
  }
  // at most one CTA per SM, at least 8 tokens each
  uint32_t n = (T + 7) / 8;
  if (n > sms) n = sms;
  *per = (T + n - 1) / n;
  *grid = (T + *per - 1) / *per;
}

template <int NPER>
cudaError_t run_route(const GrArgs &a, uint32_t grid, cudaStream_t stream) {
  auto kern = k_group_route<NPER>;
  const uint32_t E = a.r.n_expert;
  const bool few = grid == 1 && a.T * a.r.top_k <= kGrFewRows;
  // few rows: a warp a token, and enough of them to write off[]
  const uint32_t threads = few ? 32 * (a.T > 8 ? a.T : 8) : kGrThreads;
  const size_t smem = 4 * ((size_t)kGrWarps * 32 + threads * NPER +
                           (few ? 0 : (size_t)E * (kGrMaskWords + 1) + 32));
  static int set[kMaxDevices];
  const cudaError_t e = allow_smem(kern, smem, set);
  if (e != cudaSuccess) return e;
  if (grid == 1) return launch_k(kern, 1, threads, smem, stream, true, a, few);
  GrArgs args = a;
  bool no = false;
  void *p[] = {&args, &no};
  return cudaLaunchCooperativeKernel((const void *)kern, dim3(grid), dim3(kGrThreads), p, smem,
                                     stream);
}

}  // namespace

size_t group_route_ws(const moe_router &r, uint32_t T) {
  (void)T;
  return MOE_WS_FIXED_BYTES + (size_t)kFp8MaxCtas * r.n_expert * 4;
}

cudaError_t launch_group_route(const moe_router &r, const void *logits, int dt, size_t ld,
                               const float *bias, uint32_t T, int32_t *idx, float *w,
                               int32_t *off, int32_t *perm, int32_t *pos, void *ws,
                               cudaStream_t stream) {
  GrArgs a;
  a.r = r;
  a.logits = logits;
  a.dt = dt;
  a.ld = ld;
  a.bias = bias;
  a.T = T;
  a.gsize = r.n_expert / r.n_group;
  a.idx = idx;
  a.w = w;
  a.off = off;
  a.perm = perm;
  a.pos = pos;
  a.hist = (int32_t *)((uint8_t *)ws + MOE_WS_FIXED_BYTES);
  a.sync = (uint32_t *)((uint8_t *)ws + 256) + kFp8RouteSync;
  a.err = (uint32_t *)ws;
  uint32_t grid;
  gr_split(T, (uint32_t)fp8_ctas(), &a.per_cta, &grid);
  const uint32_t nper = (r.n_expert + 31) / 32;
  if (nper <= 1) return run_route<1>(a, grid, stream);
  if (nper <= 2) return run_route<2>(a, grid, stream);
  if (nper <= 4) return run_route<4>(a, grid, stream);
  if (nper <= 5) return run_route<5>(a, grid, stream);
  if (nper <= 8) return run_route<8>(a, grid, stream);
  if (nper <= 12) return run_route<12>(a, grid, stream);
  if (nper <= 16) return run_route<16>(a, grid, stream);
  return run_route<32>(a, grid, stream);
}

}  // namespace moe
