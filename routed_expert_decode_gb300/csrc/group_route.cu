// group_route.cu -- group-limited top-k routing and the stable permutation of
// the (token, slot) rows by expert.
//
// Many tokens: a warp selects for a token, and a second kernel permutes.
// The token's logits go to shared memory, where one rolled loop turns them into
// selection values c (unrolled over a lane's experts the code is ten times as long,
// and runs from a cold instruction cache).  Then lane l holds the NPER consecutive
// experts [l*NPER, (l+1)*NPER), so "lowest index" is "lowest lane, then lowest
// register" and a group of experts is a run of lanes: where the group size is NPER
// times a power of two, a group's best two c meet by shuffles inside the run; other
// sizes are scanned in shared memory.  Scores become order-preserving unsigned
// keys; a round of top-k is one redux.sync maximum and one ballot (the lowest lane
// that holds it wins); the winner goes on to its second-best, and looks through its
// registers again only when that is used up.
//
// Permutation: up to 64 CTAs, each with a run of the tokens.  The selecting warps count
// the picks of each run per expert (in counters that a kernel before them clears), and
// a CTA adds up the counts of the runs before its own and of the experts before
// each expert: where its rows of each expert start.  A token picks an expert at
// most once, so the rank of row (t, j) among its expert's rows of a run of tokens is a
// population count over the expert's token mask below bit t.  No order of atomics
// enters the result, and no CTA waits for another.
//
// Few rows: one CTA, a thread for each expert of a token: an expert's place is the
// number of kept ones before it, so there are no rounds; rows are ranked by
// comparing them all.
//
// What bounds it: for many tokens the selection's issue slots (256 experts, top 8:
// ~1100 warp instructions a token; the logits are read once) and the fixed steps of
// the permutation (two launches and two passes over its picks, ~5 us); for few tokens
// the chain of a launch and its dependent steps.  256 experts in 8 groups, 4 kept, top
// 8: 8192 tokens 21.0 us, 256 tokens 9.7, 32 tokens 7.5, one 5.1.  A permutation that
// counted by itself behind a grid-wide barrier: 22.6 and 11.2 us for 8192 and 256.
#include "router_math.cuh"

namespace moe {
namespace {

constexpr int kGrWarps = 4;  // tokens of a selecting CTA (64 tokens: 7.4 us, 7.6 with 8)
// A call of one or two tokens runs on k_group_few (256 experts: 5.1 and 5.8 us; 7.7
// with four tokens, 7.0 on the two kernels).
constexpr uint32_t kGrFewTokens = 2;
constexpr int kGrFewThreads = 1024;
constexpr int kPlaceThreads = 1024;
// The permutation's CTAs: few enough that adding up their counts is cheap, enough
// that their scattered stores are (8192 tokens: 64 CTAs, see k_group_place)
constexpr uint32_t kPlaceCtas = 64;
constexpr uint32_t kPlaceWords = 4;                  // mask words of an expert
constexpr uint32_t kPlaceTokens = 32 * kPlaceWords;  // tokens ranked at a time

struct GrArgs {
  moe_router r;
  const void *logits;
  int dt;
  size_t ld;
  const float *bias;
  uint32_t T, gsize;  // experts per group
  int32_t *idx;
  float *w;
  int32_t *off, *perm, *pos;
  int32_t *hist;          // [runs][E] picks of each run's tokens, or null (one run)
  uint32_t per, per_inv;  // tokens of a run, floor((2^32 - 1) / per)
};

// The arguments into the constant cache before the wait for earlier work: a
// launch's are always cold, and the first uses come one after another.
__device__ __forceinline__ void gr_warm(const GrArgs &a) {
  asm volatile("" ::"r"(a.r.n_expert), "r"(a.r.top_k), "r"(a.r.n_group), "r"(a.r.topk_group),
               "r"(a.r.score), "r"(a.r.group_score), "r"(a.r.renorm), "f"(a.r.s), "l"(a.logits),
               "r"(a.dt), "l"(a.ld), "l"(a.bias), "r"(a.T), "r"(a.gsize), "l"(a.idx), "l"(a.w),
               "l"(a.off), "l"(a.perm), "l"(a.pos), "l"(a.hist), "r"(a.per), "r"(a.per_inv));
}

// order-preserving map of a float (never NaN) to an unsigned above 0; -0 as +0
__device__ __forceinline__ uint32_t order_key(float c) {
  const uint32_t b = __float_as_uint(c + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ float load_logit(const void *p, int dt, size_t i) {
  float v;
  if (dt == MOE_DT_F32) v = ((const float *)p)[i];
  else if (dt == MOE_DT_BF16) v = __bfloat162float(((const __nv_bfloat16 *)p)[i]);
  else v = __half2float(((const __half *)p)[i]);
  return logit_value(v);
}
// fn(logit, expert) of a token's E logits to shared memory, by its warp
template <int DT, typename F>
__device__ __forceinline__ void stage_token(const void *p, size_t row, uint32_t E, int lane,
                                            float *sc, const F &fn) {
  const typename Elem<DT>::T *src = (const typename Elem<DT>::T *)p + row;
#pragma unroll 4
  for (uint32_t i = lane; i < E; i += 32) sc[i] = fn(logit_value(Elem<DT>::to(src[i])), i);
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

// One token by one warp: its picks to idx and w.  sc: 32 * NPER floats of shared
// memory of the warp.
template <int NPER>
__device__ __forceinline__ void route_token(const GrArgs &a, uint32_t t, int lane, float *sc) {
  const uint32_t E = a.r.n_expert, k = a.r.top_k, G = a.r.n_group;
  const uint32_t e0 = (uint32_t)lane * NPER;
  const size_t row = (size_t)t * a.ld;
  const uint32_t fn = a.r.score;
  auto stage = [&](const auto &f) {
    if (a.dt == MOE_DT_F32) stage_token<MOE_DT_F32>(a.logits, row, E, lane, sc, f);
    else if (a.dt == MOE_DT_BF16) stage_token<MOE_DT_BF16>(a.logits, row, E, lane, sc, f);
    else stage_token<MOE_DT_F16>(a.logits, row, E, lane, sc, f);
  };
  auto biased = [&](float p, uint32_t e) { return a.bias ? no_nan(p + a.bias[e]) : p; };
  float m = -INFINITY, rsum = 0.0f;  // softmax: the row's maximum and 1 / sum
  if (fn == MOE_SCORE_SIGMOID) {
    stage([&](float l, uint32_t e) { return biased(sigmoid_of(l), e); });
  } else if (fn == MOE_SCORE_SQRT_SOFTPLUS) {
    stage([&](float l, uint32_t e) { return biased(softplus_root_of(l), e); });
  } else {
    stage([&](float l, uint32_t) {
      m = fmaxf(m, l);
      return l;
    });
    m = key_value(__reduce_max_sync(0xffffffffu, order_key(m)));
    float sum = 0.0f;
    for (uint32_t i = lane; i < E; i += 32) sum += softmax_term(sc[i], m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    rsum = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
    if (a.bias || a.r.group_score != MOE_GROUP_MAX)  // else selection is by what is staged
      for (uint32_t i = lane; i < E; i += 32) sc[i] = biased(softmax_term(sc[i], m) * rsum, i);
  }
  auto score = [&](float l) {
    return fn == MOE_SCORE_SIGMOID ? sigmoid_of(l)
           : fn == MOE_SCORE_SOFTMAX ? softmax_term(l, m) * rsum : softplus_root_of(l);
  };
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
    const bool runs = gs % NPER == 0 && (run & (run - 1)) == 0;
    float mine = -INFINITY;  // lane g: the score of group g
    if (runs) {
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
    if (runs) {  // a lane's experts are of one group
      if (!((kept >> ((uint32_t)lane >> (31 - __clz(run)))) & 1u)) {
#pragma unroll
        for (int i = 0; i < NPER; ++i) key[i] = 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NPER; ++i)
        if (e0 + i < E && !((kept >> ((e0 + i) / gs)) & 1u)) key[i] = 0u;
    }
  }
  // ---- top k: a lane's two best keys and the first registers that hold them; of
  // equal keys the lower register comes first
  uint32_t best = 0u, next = 0u;
  int at = 0, at2 = 0;
  uint32_t used = 0u;  // registers that were picked
  auto look = [&](bool again) {
    best = next = 0u;
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const uint32_t v = again && ((used >> i) & 1u) ? 0u : key[i];
      const bool first = v > best, second = v > next;
      next = first ? best : second ? v : next;
      at2 = first ? at : second ? i : at2;
      best = first ? v : best;
      at = first ? i : at;
    }
  };
  look(false);
  // the staged values are not needed any more: the picks in their place
  int *pick = (int *)sc;
  __syncwarp();
#pragma unroll 1
  for (uint32_t j = 0; j < k; ++j) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const int win = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
    if (lane == win) {
      pick[j] = (int)e0 + at;
      used |= 1u << at;
      if (next == 0u) {
        look(true);
      } else {
        best = next;
        at = at2;
        next = 0u;
      }
    }
  }
  __syncwarp();
  // ---- weights: lane j evaluates its pick's p again from the logit
  const bool slot = (uint32_t)lane < k;
  const int mine = slot ? pick[lane] : 0;
  const float p = slot ? score(load_logit(a.logits, a.dt, row + mine)) : 0.0f;
  float w = a.r.s * p;
  if (a.r.renorm) {
    float sum = p;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f;
  }
  if (slot) {
    a.idx[(size_t)t * k + lane] = mine;
    a.w[(size_t)t * k + lane] = w;
    if (a.hist) atomicAdd(a.hist + (size_t)quotient(t, a.per, a.per_inv) * E + mine, 1);
  }
}

template <int NPER>
__global__ void __launch_bounds__(kGrWarps * 32) k_group_route(const GrArgs a) {
  pdl_trigger();
  gr_warm(a);
  pdl_wait();
  __shared__ __align__(16) float sc[kGrWarps][32 * NPER];
  const int warp = threadIdx.x >> 5;
  const uint32_t t = blockIdx.x * kGrWarps + warp;
  if (t < a.T) route_token<NPER>(a, t, threadIdx.x & 31, sc[warp]);
}

__global__ void __launch_bounds__(1024) k_group_clear(int32_t *hist, uint32_t n) {
  pdl_trigger();
  pdl_wait();
  for (uint32_t i = blockIdx.x * 1024 + threadIdx.x; i < n; i += gridDim.x * 1024) hist[i] = 0;
}

struct PlaceArgs {
  const int32_t *idx;
  uint32_t T, per, k, k_inv, E;  // per: tokens of a CTA; k_inv = floor((2^32 - 1) / k)
  int32_t *off, *perm, *pos;
  const int32_t *hist;  // [CTAs][E]: rows of each CTA's tokens per expert
};

// off, perm and pos: CTA c places the rows of tokens [c*per, (c+1)*per)
__global__ void __launch_bounds__(kPlaceThreads) k_group_place(const PlaceArgs a) {
  pdl_trigger();
  asm volatile("" ::"l"(a.idx), "r"(a.T), "r"(a.per), "r"(a.k), "r"(a.k_inv), "r"(a.E), "l"(a.off),
               "l"(a.perm), "l"(a.pos), "l"(a.hist));
  extern __shared__ __align__(16) uint8_t psm[];
  const uint32_t E = a.E, k = a.k, c = blockIdx.x;
  uint32_t *mask = (uint32_t *)psm;             // [E][words]
  int *count = (int *)(mask + E * kPlaceWords);  // [E]: this CTA's rows, then its next row
  __shared__ int red[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t t0 = min(a.T, c * a.per), t1 = min(a.T, t0 + a.per);
  for (uint32_t e = tid; e < E; e += kPlaceThreads) count[e] = 0;
  __syncthreads();
  pdl_wait();
  // the picks of tokens [x, y), as (expert, pick within the run)
  auto each = [&](uint32_t x, uint32_t y, auto &&use) {
    const uint32_t n = (y - x) * k;
    const int32_t *p = a.idx + (size_t)x * k;
    for (uint32_t i = tid; i < n; i += kPlaceThreads) use(p[i], i);
  };
  auto token_of = [&](uint32_t i) { return quotient(i, k, a.k_inv); };
  int all = 0, ahead = 0;  // thread e: rows of expert e, and those of earlier CTAs
  if (gridDim.x == 1) {
    each(t0, t1, [&](int e, uint32_t) { atomicAdd(&count[e], 1); });
    __syncthreads();
    if ((uint32_t)tid < E) all = count[tid];
  } else {
    // kPlaceThreads / E threads an expert share the runs' counts
    int *part = (int *)mask;  // [2][E], free until the ranking
    for (uint32_t e = tid; e < 2 * E; e += kPlaceThreads) part[e] = 0;
    __syncthreads();
    const uint32_t lanes = (uint32_t)kPlaceThreads / E;
    const uint32_t e = (uint32_t)tid % E, p = (uint32_t)tid / E;
    if (p < lanes) {
      int b = 0, s = 0;
#pragma unroll 16
      for (uint32_t q = p; q < gridDim.x; q += lanes) {
        const int v = __ldcg(a.hist + (size_t)q * E + e);
        s += v;
        b += q < c ? v : 0;
      }
      atomicAdd(&part[e], s);  // integer sums: any order gives the same
      atomicAdd(&part[E + e], b);
    }
    __syncthreads();
    if ((uint32_t)tid < E) {
      all = part[tid];
      ahead = part[E + tid];
    }
  }
  // exclusive scan over the experts
  int incl = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) red[warp] = incl;
  __syncthreads();
  {
    int v = red[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    const int first = incl - all + (warp > 0 ? __shfl_sync(0xffffffffu, v, warp - 1) : 0);
    if ((uint32_t)tid < E) {
      if (c == 0) {
        a.off[tid] = first;
        if ((uint32_t)tid == E - 1) a.off[E] = first + all;
      }
      count[tid] = first + ahead;
    }
  }
  for (uint32_t r0 = t0; r0 < t1; r0 += kPlaceTokens) {
    const uint32_t r1 = min(t1, r0 + kPlaceTokens);
    for (uint32_t i = tid; i < E * kPlaceWords; i += kPlaceThreads) mask[i] = 0u;
    __syncthreads();
    each(r0, r1, [&](int e, uint32_t i) {
      const uint32_t t = token_of(i);
      atomicOr(&mask[e * kPlaceWords + (t >> 5)], 1u << (t & 31));
    });
    __syncthreads();
    each(r0, r1, [&](int e, uint32_t i) {
      const uint32_t t = token_of(i), w = t >> 5;
      const uint32_t *m = mask + e * kPlaceWords;
      int row = count[e] + __popc(m[w] & ((1u << (t & 31)) - 1u));
#pragma unroll
      for (uint32_t q = 0; q + 1 < kPlaceWords; ++q) row += q < w ? __popc(m[q]) : 0;
      const size_t r = (size_t)r0 * k + i;
      a.perm[row] = (int32_t)r;
      a.pos[r] = row;
    });
    __syncthreads();
    for (uint32_t e = tid; e < E; e += kPlaceThreads) {
      int n = 0;
#pragma unroll
      for (uint32_t q = 0; q < kPlaceWords; ++q) n += __popc(mask[e * kPlaceWords + q]);
      count[e] += n;
    }
    __syncthreads();
  }
}

// A call of few rows: a team of threads per token, a thread an expert.
__global__ void __launch_bounds__(kGrFewThreads) k_group_few(const GrArgs a, const uint32_t team) {
  pdl_trigger();
  gr_warm(a);
  pdl_wait();
  __shared__ __align__(16) uint32_t keys[kGrFewThreads];
  __shared__ uint32_t gkey[kGrFewThreads];             // [teams][32]: the groups' keys
  __shared__ float wred[32];                           // a warp's partial results
  __shared__ int pick[kGrFewTokens][32];
  __shared__ float pick_p[kGrFewTokens][32];
  const uint32_t E = a.r.n_expert, k = a.r.top_k, G = a.r.n_group, gs = a.gsize;
  const uint32_t fn = a.r.score;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t m = (uint32_t)tid / team, e = (uint32_t)tid - m * team;  // team, expert
  const uint32_t teams = blockDim.x / team, w0 = m * (team / 32), nw = team / 32;
  uint32_t *tk = keys + m * team;
  for (uint32_t t0 = 0; t0 < a.T; t0 += teams) {
    const uint32_t t = t0 + m;
    const bool live = t < a.T && e < E;
    const float l = live ? load_logit(a.logits, a.dt, (size_t)t * a.ld + e) : -INFINITY;
    const float b = live && a.bias ? a.bias[e] : 0.0f;
    float p;
    if (fn == MOE_SCORE_SOFTMAX) {
      const uint32_t wk = __reduce_max_sync(0xffffffffu, order_key(l));
      if (lane == 0) wred[warp] = key_value(wk);
      __syncthreads();
      float mx = -INFINITY;
      for (uint32_t i = 0; i < nw; ++i) mx = fmaxf(mx, wred[w0 + i]);
      const float x = softmax_term(l, mx);
      float sum = x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      __syncthreads();
      if (lane == 0) wred[warp] = sum;
      __syncthreads();
      sum = 0.0f;
      for (uint32_t i = 0; i < nw; ++i) sum += wred[w0 + i];
      p = x * (sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f);
    } else {
      p = fn == MOE_SCORE_SIGMOID ? sigmoid_of(l) : softplus_root_of(l);
    }
    const bool by_logit =
        fn == MOE_SCORE_SOFTMAX && !a.bias && a.r.group_score == MOE_GROUP_MAX;
    uint32_t key = live ? order_key(by_logit ? l : a.bias ? no_nan(p + b) : p) : 0u;
    tk[e] = key;
    uint32_t kept = 0xffffffffu;  // groups
    __syncthreads();
    if (a.r.topk_group < G) {
      // a warp a group: its two best
      for (uint32_t g = warp - w0; g < G; g += nw) {
        uint32_t b1 = 0u, b2 = 0u;
        for (uint32_t i = lane; i < gs; i += 32) {
          const uint32_t v = tk[g * gs + i];
          b2 = max(b2, min(b1, v));
          b1 = max(b1, v);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const uint32_t p1 = __shfl_xor_sync(0xffffffffu, b1, o);
          const uint32_t p2 = __shfl_xor_sync(0xffffffffu, b2, o);
          b2 = max(max(b2, p2), min(b1, p1));
          b1 = max(b1, p1);
        }
        const bool two = a.r.group_score == MOE_GROUP_TOP2_SUM && gs > 1;
        if (lane == 0)
          gkey[m * 32 + g] =
              two ? order_key(no_nan(key_value(b1) + key_value(b2))) : b1;
      }
      __syncthreads();
      const uint32_t gk = (uint32_t)lane < G ? gkey[m * 32 + lane] : 0u;
      uint32_t ahead = 0;  // groups that go before this lane's
      for (uint32_t g = 0; g < G; ++g) {
        const uint32_t ok = __shfl_sync(0xffffffffu, gk, g);
        ahead += ok > gk || (ok == gk && g < (uint32_t)lane);
      }
      kept = __ballot_sync(0xffffffffu, (uint32_t)lane < G && ahead < a.r.topk_group);
    }
    // an expert's place: the kept ones before it
    const uint32_t mine = G == 1 ? 0u : e / gs;
    if (live && ((kept >> mine) & 1u)) {
      uint32_t place = 0;
      for (uint32_t g = 0; g < G; ++g) {
        if (!((kept >> g) & 1u)) continue;
        const uint32_t g0 = g * gs, g1 = g0 + gs;
        uint32_t i = g0;
        if ((g0 & 3u) == 0)
#pragma unroll 4
          for (; i + 4 <= g1; i += 4) {
            const uint4 v = *(const uint4 *)(tk + i);
            place += v.x > key || (v.x == key && i < e);
            place += v.y > key || (v.y == key && i + 1 < e);
            place += v.z > key || (v.z == key && i + 2 < e);
            place += v.w > key || (v.w == key && i + 3 < e);
          }
        for (; i < g1; ++i) place += tk[i] > key || (tk[i] == key && i < e);
      }
      if (place < k) {
        pick[t][place] = (int)e;
        pick_p[t][place] = p;
      }
    }
    __syncthreads();
    if (t < a.T && e < 32) {  // the team's first warp
      const bool slot = e < k;
      const float pj = slot ? pick_p[t][e] : 0.0f;
      float w = a.r.s * pj;
      if (a.r.renorm) {
        float sum = pj;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        w = sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f;
      }
      if (slot) {
        a.idx[(size_t)t * k + e] = pick[t][e];
        a.w[(size_t)t * k + e] = w;
      }
    }
  }
  for (uint32_t x = tid; x <= E; x += blockDim.x) {
    int n = 0;
    for (uint32_t t = 0; t < a.T; ++t)
#pragma unroll 8
      for (uint32_t j = 0; j < k; ++j) n += pick[t][j] < (int)x;
    a.off[x] = n;
  }
  for (uint32_t r = tid; r < a.T * k; r += blockDim.x) {
    const uint32_t tr = r / k;
    const int x = pick[tr][r - tr * k];
    int row = 0;
    for (uint32_t t = 0; t < a.T; ++t)
#pragma unroll 8
      for (uint32_t j = 0; j < k; ++j) {
        const int v = pick[t][j];
        row += v < x || (v == x && t < tr);
      }
    a.perm[row] = (int32_t)r;
    a.pos[r] = row;
  }
}

template <int NPER>
cudaError_t run_route(const GrArgs &a, cudaStream_t stream) {
  return launch_k(k_group_route<NPER>, (a.T + kGrWarps - 1) / kGrWarps, kGrWarps * 32, 0, stream,
                  true, a);
}

cudaError_t launch_select(const GrArgs &a, cudaStream_t stream) {
  const uint32_t nper = (a.r.n_expert + 31) / 32;
  if (nper <= 1) return run_route<1>(a, stream);
  if (nper <= 2) return run_route<2>(a, stream);
  if (nper <= 4) return run_route<4>(a, stream);
  if (nper <= 5) return run_route<5>(a, stream);
  if (nper <= 8) return run_route<8>(a, stream);
  if (nper <= 12) return run_route<12>(a, stream);
  if (nper <= 16) return run_route<16>(a, stream);
  return run_route<32>(a, stream);
}

}  // namespace

size_t group_route_ws(const moe_router &r) {
  return MOE_WS_FIXED_BYTES + (size_t)kPlaceCtas * r.n_expert * 4;
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
  a.hist = nullptr;
  a.per = a.per_inv = 0;
  if (T <= kGrFewTokens) {
    const uint32_t team = (r.n_expert + 31) / 32 * 32;
    const uint32_t teams = T < kGrFewThreads / team ? (T ? T : 1) : kGrFewThreads / team;
    return launch_k(k_group_few, 1, team * teams, 0, stream, true, a, team);
  }
  // a run of 128 tokens a CTA of the permutation, more once there are 64
  uint32_t grid = (T + kPlaceTokens - 1) / kPlaceTokens;
  if (grid > kPlaceCtas) grid = kPlaceCtas;
  a.per = (T + grid - 1) / grid;
  a.per_inv = 0xffffffffu / a.per;
  cudaError_t e = cudaSuccess;
  if (grid > 1) {
    a.hist = (int32_t *)((uint8_t *)ws + MOE_WS_FIXED_BYTES);
    const uint32_t n = grid * r.n_expert;
    e = launch_k(k_group_clear, (n + 4095) / 4096, 1024, 0, stream, true, a.hist, n);
    if (e != cudaSuccess) return e;
  }
  e = launch_select(a, stream);
  if (e != cudaSuccess) return e;
  PlaceArgs p;
  p.idx = idx;
  p.T = T;
  p.per = a.per;
  p.k = r.top_k;
  p.k_inv = 0xffffffffu / r.top_k;
  p.E = r.n_expert;
  p.off = off;
  p.perm = perm;
  p.pos = pos;
  p.hist = a.hist;
  const size_t smem = (size_t)p.E * (kPlaceWords + 1) * 4;
  return launch_k(k_group_place, grid, kPlaceThreads, smem, stream, true, p);
}

}  // namespace moe
