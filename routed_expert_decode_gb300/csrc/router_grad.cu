// router_grad.cu -- the loss that evens out the experts' load, and the gradients that
// reach a router's logits.
//
// A token's E logits lie on a team of lanes, 8 consecutive ones a lane and chunk (one
// 16-byte load of a 16-bit type): 8 lanes for 64 experts, so four tokens a warp, 32
// for 256 and more.  Sums over a token are shuffles inside its team.
#include "router_grad.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr uint32_t kAll = 0xffffffffu;

struct Team {
  uint32_t lanes;  // a power of two; NC > 1 chunks only with 32
  int l, t;        // lane within the team, team within the warp
  __device__ __forceinline__ uint32_t per_warp() const { return 32 / lanes; }
  __device__ __forceinline__ uint32_t expert(int c) const { return (c * lanes + l) * 8; }
  __device__ __forceinline__ float sum(float v) const {
    for (uint32_t o = 1; o < lanes; o <<= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
  }
  __device__ __forceinline__ float max(float v) const {
    for (uint32_t o = 1; o < lanes; o <<= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
  }
};

// the largest chunks' count of an expert count, and a team's lanes
inline int chunks_of(uint32_t E) { return E <= 256 ? 1 : E <= 512 ? 2 : 4; }
inline uint32_t team_lanes(uint32_t E) {
  uint32_t n = 1;
  while (n < 32 && n * 8 < E) n *= 2;
  return n;
}
__device__ __forceinline__ Team team_here(uint32_t lanes) {
  const int lane = threadIdx.x & 31;
  Team t;
  t.lanes = lanes;
  t.l = lane & (int)(lanes - 1);
  t.t = lane / (int)lanes;
  return t;
}

// One token's logits; lanes and elements without an expert hold -inf, whose score is 0.
template <int DT, int NC>
struct Row {
  Raw8<DT> raw[NC];
  __device__ __forceinline__ void load(const void *base, size_t ld, uint32_t t, uint32_t E,
                                       const Team &tm, bool vec, bool live) {
    using X = Elem<DT>;
    const typename X::T *row = (const typename X::T *)base + (size_t)t * ld;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const uint32_t e = tm.expert(c);
      if (vec && live && e < E) {
        raw[c].load(row + e);
      } else {
        typename X::T *v = (typename X::T *)raw[c].v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = live && e + i < E ? row[e + i] : X::from(-INFINITY);
      }
    }
  }
  __device__ __forceinline__ void to(float (&l)[NC][8]) const {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      raw[c].to(l[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) l[c][i] = logit_value(l[c][i]);
    }
  }
};

// l -> scores p (softmax: whose sum is 1), in place; slope = d log p / dl, softmax's
// without its sum's part.  Returns the sum of p.
template <int NC, bool SLOPE>
__device__ __forceinline__ float scores(uint32_t fn, const Team &tm, float (&l)[NC][8],
                                        float (&slope)[NC][8]) {
  float s = 0.0f;
  if (fn == MOE_SCORE_SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, l[c][i]);
    m = tm.max(m);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        l[c][i] = softmax_term(l[c][i], m);
        s += l[c][i];
        if (SLOPE) slope[c][i] = 1.0f;
      }
    s = tm.sum(s);
    const float r = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) l[c][i] *= r;
    return s > 0.0f ? 1.0f : 0.0f;
  }
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // of e^-|l|: 1/(1+e) is the larger of sigmoid(l) and sigmoid(-l), e/(1+e) the other
      const float v = l[c][i], e = expf(-fabsf(v));
      const float big = __frcp_rn(1.0f + e), small = e * big;
      const float up = v >= 0.0f ? big : small;
      if (fn == MOE_SCORE_SIGMOID) {
        l[c][i] = up;
        if (SLOPE) slope[c][i] = v >= 0.0f ? small : big;
      } else {
        const float soft = fmaxf(v, 0.0f) + log1pf(e);
        l[c][i] = __fsqrt_rn(soft);
        // sigmoid / (2 softplus); 1/2 in the limit of -inf
        if (SLOPE) slope[c][i] = soft > 0.0f ? __fdiv_rn(0.5f * up, soft) : 0.5f;
      }
      s += l[c][i];
    }
  return tm.sum(s);
}

// ---------------------------------------------------------------- sequences
__device__ __forceinline__ int seq_at(const moe_tokens &t, uint32_t s) {
  return t.seq ? min(max(t.seq[s], 0), (int)t.T) : s == 0 ? 0 : (int)t.T;
}
// the first sequence that ends behind token x (S: none)
__device__ __forceinline__ uint32_t seq_of(const moe_tokens &t, int x) {
  uint32_t lo = 0, hi = t.S;
  while (lo < hi) {
    const uint32_t mid = (lo + hi) / 2;
    if (seq_at(t, mid + 1) > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// ---------------------------------------------------------------- the loss
// CTA c has tokens [c*per, (c+1)*per), whatever sequences they are of.  What it
// adds up of a sequence that lies within them it finishes itself; of one that goes on
// before or behind, the sums go to the workspace (the first slot if the sequence begins
// before the CTA's tokens, the second if it begins among them: at most one each), where
// k_balance_join adds them in order.
constexpr uint32_t kSumCtas = 304;  // two an SM, at most
constexpr uint32_t kSumTokens = 64;  // tokens of a CTA, at least

struct BalanceArgs {
  RouterGradArgs g;
  uint32_t lanes, per;
  bool vec;
  int32_t *count, *tokens;
  float *prob, *loss;
  float *part;         // [CTAs][2][E] sums of shares
  int32_t *part_count;  // [CTAs][2][E] picks
  int32_t *part_n;      // [CTAs][2] counting tokens
  float *seq_loss;     // [S]
  uint32_t *ticket;
};

// sum over the block's threads in a fixed order, to all of them; red: 32 floats
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) v += red[i];
  return v;
}

// a sequence's outputs from its sums; n, picks(e) and shares(e) as summed
template <int THREADS, typename C, typename P>
__device__ __forceinline__ void finish_sequence(const BalanceArgs &a, uint32_t s, int n, float *red,
                                                const C &picks, const P &shares) {
  const uint32_t E = a.g.r.n_expert;
  float loss = 0.0f;
  for (uint32_t e = threadIdx.x; e < E; e += THREADS) {
    const int c = picks(e);
    const float p = n > 0 ? __fdiv_rn(shares(e), (float)n) : 0.0f;
    a.count[(size_t)s * E + e] = c;
    a.prob[(size_t)s * E + e] = p;
    loss += (float)c * p;
  }
  loss = block_sum<THREADS>(loss, red);
  if (threadIdx.x == 0) {
    a.tokens[s] = n;
    a.seq_loss[s] =
        n > 0 ? loss * __fdiv_rn((float)E, (float)a.g.r.top_k * (float)n) : 0.0f;
  }
}

// the loss from the sequences' terms, by one block
template <int THREADS>
__device__ __forceinline__ void finish_loss(const BalanceArgs &a, float *red) {
  float v = 0.0f;
  for (uint32_t s = threadIdx.x; s < a.g.t.S; s += THREADS) v += __ldcg(a.seq_loss + s);
  v = block_sum<THREADS>(v, red);
  if (threadIdx.x == 0) a.loss[0] = v * __fdiv_rn(a.g.coef, (float)a.g.t.S);
}

template <int DT, int NC>
__global__ void __launch_bounds__(kThreads) k_balance(const BalanceArgs a) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ __align__(16) uint8_t bsm[];
  const uint32_t E = a.g.r.n_expert, k = a.g.r.top_k;
  const uint32_t width = NC * a.lanes * 8;
  float *red = (float *)bsm;                     // [kWarps][width]
  int *cnt = (int *)(red + kWarps * width);      // [width]
  __shared__ float sums[32];
  __shared__ int live_n;
  const int tid = threadIdx.x, warp = tid >> 5;
  const Team tm = team_here(a.lanes);
  const bool alone = gridDim.x == 1;
  const int t0 = (int)min(a.g.t.T, blockIdx.x * a.per);
  const int t1 = (int)min((uint64_t)a.g.t.T, (uint64_t)t0 + a.per);
  constexpr int U = NC == 1 ? 4 : 2;  // tokens of a team on the way together
  const int step = kWarps * (int)tm.per_warp();
  for (uint32_t s = alone ? 0 : seq_of(a.g.t, t0); s < a.g.t.S; ++s) {
    const int s0 = seq_at(a.g.t, s), s1 = seq_at(a.g.t, s + 1);
    if (!alone && s0 >= t1) break;
    const int lo = max(s0, t0), hi = min(s1, t1);
    if (lo >= hi && !alone) continue;
    for (uint32_t e = tid; e < width; e += kThreads) cnt[e] = 0;
    if (tid == 0) live_n = 0;
    __syncthreads();
    // ---- shares
    float acc[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[c][i] = 0.0f;
    for (int base = lo + warp * (int)tm.per_warp(); base < hi; base += U * step) {
      Row<DT, NC> row[U];
      bool on[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = base + u * step + tm.t;
        on[u] = t < hi && (!a.g.t.live || a.g.t.live[t]);
        row[u].load(a.g.logits, a.g.ld, (uint32_t)t, E, tm, a.vec, on[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float l[NC][8];
        row[u].to(l);
        const float sum = scores<NC, false>(a.g.r.score, tm, l, l);
        const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[c][i] = __fmaf_rn(l[c][i], inv, acc[c][i]);
      }
    }
    // ---- picks
    int mine = 0;
    if (a.g.t.live)
      for (int t = lo + tid; t < hi; t += kThreads) mine += a.g.t.live[t] != 0;
    else if (tid == 0)
      mine = max(hi - lo, 0);
    if (mine) atomicAdd(&live_n, mine);
    const uint32_t i1 = (uint32_t)max(hi, lo) * k;
#pragma unroll 4
    for (uint32_t i = (uint32_t)lo * k + tid; i < i1; i += kThreads) {
      const uint32_t e = (uint32_t)a.g.idx[i];
      if (e < E && (!a.g.t.live || a.g.t.live[i / k])) atomicAdd(&cnt[e], 1);
    }
    // ---- the warps' shares in order
    for (uint32_t o = tm.lanes; o < 32; o <<= 1)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[c][i] += __shfl_xor_sync(kAll, acc[c][i], o);
    if (tm.t == 0)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) red[warp * width + tm.expert(c) + i] = acc[c][i];
    __syncthreads();
    auto shares = [&](uint32_t e) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += red[w * width + e];
      return v;
    };
    if (s0 >= t0 && s1 <= t1) {
      finish_sequence<kThreads>(a, s, live_n, sums, [&](uint32_t e) { return cnt[e]; }, shares);
    } else {
      const size_t slot = blockIdx.x * 2 + (s0 >= t0);
      for (uint32_t e = tid; e < E; e += kThreads) {
        a.part[slot * E + e] = shares(e);
        a.part_count[slot * E + e] = cnt[e];
      }
      if (tid == 0) a.part_n[slot] = live_n;
    }
    __syncthreads();
  }
  if (alone) {
    __threadfence_block();
    __syncthreads();
    finish_loss<kThreads>(a, sums);
  }
}

constexpr int kJoinThreads = 512;

// the sequences that no CTA had to itself, empty ones, and the loss
__global__ void __launch_bounds__(kJoinThreads) k_balance_join(const BalanceArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ float sums[32];
  __shared__ float share_g[kJoinThreads];
  __shared__ int count_g[kJoinThreads];
  __shared__ int live_n;
  __shared__ bool last;
  const uint32_t E = a.g.r.n_expert;
  const int tid = threadIdx.x;
  for (uint32_t s = blockIdx.x; s < a.g.t.S; s += gridDim.x) {
    const int s0 = seq_at(a.g.t, s), s1 = seq_at(a.g.t, s + 1);
    if (s0 >= s1) {
      finish_sequence<kJoinThreads>(a, s, 0, sums, [](uint32_t) { return 0; },
                                    [](uint32_t) { return 0.0f; });
      continue;
    }
    const uint32_t c0 = (uint32_t)s0 / a.per, c1 = (uint32_t)(s1 - 1) / a.per;
    if (c0 == c1) continue;
    // the sequence begins among the tokens of c0
    auto slot = [&](uint32_t c) { return (size_t)c * 2 + ((uint32_t)s0 >= c * a.per); };
    if (tid == 0) live_n = 0;
    __syncthreads();
    int n = 0;
    for (uint32_t c = c0 + tid; c <= c1; c += kJoinThreads) n += __ldcg(a.part_n + slot(c));
    if (n) atomicAdd(&live_n, n);
    __syncthreads();
    n = live_n;
    // groups of threads share the CTAs, for a run of experts at a time
    const uint32_t run = E < (uint32_t)kJoinThreads ? E : (uint32_t)kJoinThreads;
    const uint32_t groups = kJoinThreads / run;
    float loss = 0.0f;
    for (uint32_t e0 = 0; e0 < E; e0 += run) {
      const uint32_t g = tid / run, e = e0 + tid - g * run;
      float v = 0.0f;
      int c_sum = 0;
      if (g < groups && e < E) {
#pragma unroll 8
        for (uint32_t c = c0 + g; c <= c1; c += groups) {
          v += __ldcg(a.part + slot(c) * E + e);
          c_sum += __ldcg(a.part_count + slot(c) * E + e);
        }
      }
      __syncthreads();
      share_g[tid] = v;
      count_g[tid] = c_sum;
      __syncthreads();
      if (g == 0 && e < E) {
        for (uint32_t q = 1; q < groups; ++q) {
          v += share_g[q * run + tid];
          c_sum += count_g[q * run + tid];
        }
        const float p = n > 0 ? __fdiv_rn(v, (float)n) : 0.0f;
        a.count[(size_t)s * E + e] = c_sum;
        a.prob[(size_t)s * E + e] = p;
        loss += (float)c_sum * p;
      }
    }
    loss = block_sum<kJoinThreads>(loss, sums);
    if (tid == 0) {
      a.tokens[s] = n;
      a.seq_loss[s] =
          n > 0 ? loss * __fdiv_rn((float)E, (float)a.g.r.top_k * (float)n) : 0.0f;
    }
  }
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    if (last) atomicExch(a.ticket, 0u);
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  finish_loss<kJoinThreads>(a, sums);
}

// ---------------------------------------------------------------- the logits' gradient
struct RouteBackArgs {
  RouterGradArgs g;
  uint32_t lanes, run;  // token groups of a warp
  bool vec, vec_out;
  const float *dw;
  const int32_t *count, *tokens;
  const float *dloss;
  void *dlogits;
  int odt;
  size_t ldd;
};

template <int OT, int NC>
__device__ __forceinline__ void store_row(const RouteBackArgs &a, uint32_t t, const Team &tm,
                                          const float (&d)[NC][8]) {
  typename Elem<OT>::T *row = (typename Elem<OT>::T *)a.dlogits + (size_t)t * a.ldd;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const uint32_t e = tm.expert(c);
    if (a.vec_out) {
      if (e < a.g.r.n_expert) store8<OT>(row + e, d[c]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < a.g.r.n_expert) row[e + i] = Elem<OT>::from(d[c][i]);
    }
  }
}

// A warp takes `run` consecutive groups of tokens, the next one's logits on the way while
// it works on one.  The picks' part goes through shared memory: p is laid out there
// for the picks' lanes to fetch, then the gradient, to which they add.
template <int DT, int NC>
__global__ void __launch_bounds__(kThreads) k_route_backward(const RouteBackArgs a) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ __align__(16) uint8_t rsm[];
  const uint32_t E = a.g.r.n_expert, k = a.g.r.top_k, fn = a.g.r.score;
  const Team tm = team_here(a.lanes);
  const uint32_t width = NC * a.lanes * 8, nt = tm.per_warp();
  float *buf = (float *)rsm + ((size_t)(threadIdx.x >> 5) * nt + tm.t) * width;  // the team's
  const uint64_t g0 = ((uint64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * a.run;
  const uint64_t groups = ((uint64_t)a.g.t.T + nt - 1) / nt;
  if (g0 >= groups) return;
  const uint32_t n_groups = (uint32_t)min((uint64_t)a.run, groups - g0);
  uint32_t t = (uint32_t)(g0 * nt) + tm.t;
  const bool softmax = fn == MOE_SCORE_SOFTMAX;
  // factor of a sequence's loss gradient, up to 1 / n^2
  const float factor =
      a.count ? (a.dloss ? a.dloss[0] : 1.0f) *
                    __fdiv_rn(a.g.coef * (float)E, (float)a.g.t.S * (float)k)
              : 0.0f;
  uint32_t s = a.count ? seq_of(a.g.t, (int)t) : 0;
  int s_end = a.count && s < a.g.t.S ? seq_at(a.g.t, s + 1) : 0;
  Row<DT, NC> next;
  next.load(a.g.logits, a.g.ld, t, E, tm, a.vec, t < a.g.t.T);
  for (uint32_t i = 0; i < n_groups; ++i, t += nt) {
    const bool on = t < a.g.t.T;
    float p[NC][8], slope[NC][8];
    next.to(p);
    if (i + 1 < n_groups)
      next.load(a.g.logits, a.g.ld, t + nt, E, tm, a.vec, t + nt < a.g.t.T);
    const float sum = scores<NC, true>(fn, tm, p, slope);
    float d[NC][8];
    // ---- the loss's part
    bool counts = false;
    if (a.count && on) {
      while (s < a.g.t.S && s_end <= (int)t) {
        ++s;
        if (s < a.g.t.S) s_end = seq_at(a.g.t, s + 1);
      }
      counts = s < a.g.t.S && seq_at(a.g.t, s) <= (int)t && (!a.g.t.live || a.g.t.live[t]);
    }
    if (__any_sync(kAll, counts)) {
      const int32_t *cs = a.count + (size_t)min(s, a.g.t.S - 1) * E;
      const float n = counts ? (float)max(a.tokens[s], 1) : 1.0f;
      const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
      const float f = counts ? __fdiv_rn(factor, n * n) : 0.0f;
      float dot = 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t e = tm.expert(c) + j;
          d[c][j] = e < E ? f * (float)cs[e] : 0.0f;
          dot = __fmaf_rn(d[c][j], p[c][j] * inv, dot);
        }
      dot = tm.sum(dot);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) d[c][j] = p[c][j] * inv * (d[c][j] - dot);
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) d[c][j] = 0.0f;
    }
    // ---- the picks' part
    if (a.dw) {
      auto put = [&](const float (&v)[NC][8]) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          float4 *b = (float4 *)(buf + tm.expert(c));
          b[0] = make_float4(v[c][0], v[c][1], v[c][2], v[c][3]);
          b[1] = make_float4(v[c][4], v[c][5], v[c][6], v[c][7]);
        }
      };
      auto pick = [&](uint32_t j) {  // expert of slot j, E if it is none
        return on ? min((uint32_t)a.g.idx[(size_t)t * k + j], E) : E;
      };
      __syncwarp();
      put(p);
      __syncwarp();
      float total = 0.0f, dots = 0.0f;
      for (uint32_t j = tm.l; j < k; j += tm.lanes) {
        const uint32_t e = pick(j);
        if (e < E) {
          total += buf[e];
          dots = __fmaf_rn(buf[e], a.dw[(size_t)t * k + j], dots);
        }
      }
      total = tm.sum(total);
      dots = tm.sum(dots);
      const float inv = total > 0.0f ? __fdiv_rn(1.0f, total) : 0.0f;
      if (!a.g.r.renorm && softmax) {  // every expert's p falls as a pick's rises
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) d[c][j] = __fmaf_rn(-a.g.r.s * dots, p[c][j], d[c][j]);
      }
      // the slots in order, a round of the team's lanes at a time: a lane's own part...
      const uint32_t rounds = (k + tm.lanes - 1) / tm.lanes;
      float pk[8];  // p of this lane's picks: k <= E <= 8 lanes (256 for 32 lanes: k <= 32)
#pragma unroll
      for (uint32_t m = 0; m < 8; ++m) {
        const uint32_t j = tm.l + m * tm.lanes;
        pk[m] = 0.0f;
        if (m < rounds && j < k) {
          const uint32_t e = pick(j);
          if (e < E) pk[m] = buf[e];
        }
      }
      __syncwarp();
      put(d);
      __syncwarp();
#pragma unroll
      for (uint32_t m = 0; m < 8; ++m) {
        if (m >= rounds) break;
        const uint32_t j = tm.l + m * tm.lanes;
        const uint32_t e = j < k ? pick(j) : E;
        float v = 0.0f;
        if (e < E) {
          const float g = a.dw[(size_t)t * k + j];
          v = a.g.r.renorm ? a.g.r.s * (pk[m] * inv) * (g - dots * inv) : a.g.r.s * pk[m] * g;
        }
        // ...and the lanes one after another where two of them have the same expert
        const uint32_t key = e < E ? (uint32_t)tm.t * 1024 + e : 0x80000000u + (threadIdx.x & 31);
        const uint32_t same = __match_any_sync(kAll, key);
        uint32_t before = __popc(same & ((1u << (threadIdx.x & 31)) - 1u));
        for (uint32_t turn = 0; __any_sync(kAll, before >= turn); ++turn) {
          if (before == turn && e < E) buf[e] += v;
          __syncwarp();
        }
      }
      __syncwarp();
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float4 *b = (const float4 *)(buf + tm.expert(c));
        const float4 x = b[0], y = b[1];
        d[c][0] = x.x, d[c][1] = x.y, d[c][2] = x.z, d[c][3] = x.w;
        d[c][4] = y.x, d[c][5] = y.y, d[c][6] = y.z, d[c][7] = y.w;
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) d[c][j] *= slope[c][j];
    if (!on) continue;
    if (a.odt == MOE_DT_F32) store_row<MOE_DT_F32, NC>(a, t, tm, d);
    else if (a.odt == MOE_DT_BF16) store_row<MOE_DT_BF16, NC>(a, t, tm, d);
    else store_row<MOE_DT_F16, NC>(a, t, tm, d);
  }
}

// ---------------------------------------------------------------- combine's gradients
struct CombineBackArgs {
  const void *dy;
  size_t ldy;
  const void *o;
  size_t ldo;
  uint32_t R;
  const float *w;
  const int32_t *pos;
  uint32_t T, k, d;
  float *dw;
  void *dout;
  size_t ldd;
};

// A warp takes a slot: the dot product of two rows, and one scaled.  The warps of a
// CTA are neighbouring slots, so that dy's row is read from HBM once and from L1 by the
// others.
template <int DT, int YT, bool VEC>
__global__ void __launch_bounds__(kThreads) k_combine_backward(const CombineBackArgs a) {
  pdl_trigger();
  pdl_wait();
  using X = Elem<DT>;
  using Y = Elem<YT>;
  const int lane = threadIdx.x & 31;
  const uint64_t items = (uint64_t)a.T * a.k;
  for (uint64_t it = (uint64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); it < items;
       it += (uint64_t)gridDim.x * kWarps) {
    const uint32_t t = (uint32_t)(it / a.k);
    const uint32_t r = (uint32_t)a.pos[it];
    if (r >= a.R) {
      if (a.dw && lane == 0) a.dw[it] = 0.0f;
      continue;
    }
    const typename Y::T *y = (const typename Y::T *)a.dy + (size_t)t * a.ldy;
    const typename X::T *o = (const typename X::T *)a.o + (size_t)r * a.ldo;
    typename X::T *g = (typename X::T *)a.dout + (size_t)r * a.ldd;
    const float w = a.dout ? a.w[it] : 0.0f;
    float sum = 0.0f;
#pragma unroll 4
    for (uint32_t c = lane * 8; c < a.d; c += 256) {
      float fy[8], fo[8];
      Raw8<DT> ro;
      Raw8<YT> ry;
      if (VEC) {
        if (a.dw) ro.load(o + c);
        const uint4 *q = (const uint4 *)(y + c);
#pragma unroll
        for (int i = 0; i < (YT == MOE_DT_F32 ? 2 : 1); ++i) ry.v[i] = q[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (a.dw) ((typename X::T *)ro.v)[i] = c + i < a.d ? o[c + i] : X::from(0.0f);
          ((typename Y::T *)ry.v)[i] = c + i < a.d ? y[c + i] : Y::from(0.0f);
        }
      }
      ry.to(fy);
      if (a.dw) {
        ro.to(fo);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __fmaf_rn(fo[i], fy[i], sum);
      }
      if (a.dout) {
#pragma unroll
        for (int i = 0; i < 8; ++i) fy[i] *= w;
        if (VEC) {
          store8<DT>(g + c, fy);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < a.d) g[c + i] = X::from(fy[i]);
        }
      }
    }
    if (a.dw) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
      if (lane == 0) a.dw[it] = sum;
    }
  }
}

bool vec_rows(const void *p, int dt, size_t ld) {
  return ((uintptr_t)p & 15) == 0 && ld * dtype_size(dt) % 16 == 0;
}

template <int DT>
cudaError_t balance_t(const BalanceArgs &a, unsigned grid, cudaStream_t stream) {
  const int nc = chunks_of(a.g.r.n_expert);
  const size_t smem = (size_t)(kWarps + 1) * nc * a.lanes * 8 * 4;
  if (nc == 1) return launch_k(k_balance<DT, 1>, grid, kThreads, smem, stream, true, a);
  if (nc == 2) return launch_k(k_balance<DT, 2>, grid, kThreads, smem, stream, true, a);
  return launch_k(k_balance<DT, 4>, grid, kThreads, smem, stream, true, a);
}

template <int DT>
cudaError_t route_backward_t(const RouteBackArgs &a, unsigned grid, cudaStream_t stream) {
  const int nc = chunks_of(a.g.r.n_expert);
  const size_t smem = (size_t)kWarps * 32 / a.lanes * nc * a.lanes * 8 * 4;
  if (nc == 1) return launch_k(k_route_backward<DT, 1>, grid, kThreads, smem, stream, true, a);
  if (nc == 2) return launch_k(k_route_backward<DT, 2>, grid, kThreads, smem, stream, true, a);
  return launch_k(k_route_backward<DT, 4>, grid, kThreads, smem, stream, true, a);
}

template <int DT, int YT>
cudaError_t combine_backward_t(const CombineBackArgs &a, cudaStream_t stream) {
  const uint64_t items = (uint64_t)a.T * a.k, most = (uint64_t)fp8_ctas() * 8;
  const uint64_t need = (items + kWarps - 1) / kWarps;
  const unsigned grid = (unsigned)(need < most ? need : most);
  const bool vec = a.d % 8 == 0 && vec_rows(a.dy, YT, a.ldy) && (!a.dw || vec_rows(a.o, DT, a.ldo)) &&
                   (!a.dout || vec_rows(a.dout, DT, a.ldd));
  return launch_k(vec ? k_combine_backward<DT, YT, true> : k_combine_backward<DT, YT, false>, grid,
                  kThreads, 0, stream, true, a);
}

template <int DT>
cudaError_t combine_backward_from(int ydt, const CombineBackArgs &a, cudaStream_t stream) {
  if (ydt == MOE_DT_F32) return combine_backward_t<DT, MOE_DT_F32>(a, stream);
  if (ydt == MOE_DT_BF16) return combine_backward_t<DT, MOE_DT_BF16>(a, stream);
  return combine_backward_t<DT, MOE_DT_F16>(a, stream);
}

uint32_t balance_ctas(uint32_t T) {
  const uint32_t n = (T + kSumTokens - 1) / kSumTokens;
  return n < 1 ? 1 : n < kSumCtas ? n : kSumCtas;
}

}  // namespace

size_t balance_ws(const moe_router &r, uint32_t T, uint32_t S) {
  const size_t n = balance_ctas(T);
  return MOE_WS_FIXED_BYTES + 4 * (n * 2 * (2 * (size_t)r.n_expert + 1) + S);
}

cudaError_t launch_balance(const RouterGradArgs &g, int32_t *count, int32_t *tokens, float *prob,
                           float *loss, void *ws, cudaStream_t stream) {
  BalanceArgs a;
  a.g = g;
  const uint32_t E = g.r.n_expert, n = balance_ctas(g.t.T);
  a.lanes = team_lanes(E);
  a.per = (g.t.T + n - 1) / n;
  if (a.per == 0) a.per = 1;
  a.vec = E % 8 == 0 && vec_rows(g.logits, g.dt, g.ld);
  a.count = count;
  a.tokens = tokens;
  a.prob = prob;
  a.loss = loss;
  a.ticket = (uint32_t *)((uint8_t *)ws + 256) + kBalanceSync;
  a.part = (float *)((uint8_t *)ws + MOE_WS_FIXED_BYTES);
  a.part_count = (int32_t *)(a.part + (size_t)n * 2 * E);
  a.part_n = a.part_count + (size_t)n * 2 * E;
  a.seq_loss = (float *)(a.part_n + (size_t)n * 2);
  cudaError_t e = g.dt == MOE_DT_F32    ? balance_t<MOE_DT_F32>(a, n, stream)
                  : g.dt == MOE_DT_BF16 ? balance_t<MOE_DT_BF16>(a, n, stream)
                                        : balance_t<MOE_DT_F16>(a, n, stream);
  if (e != cudaSuccess || n == 1) return e;
  const uint32_t most = 4 * (uint32_t)fp8_ctas();
  return launch_k(k_balance_join, g.t.S < most ? g.t.S : most, kJoinThreads, 0, stream, true, a);
}

cudaError_t launch_route_backward(const RouterGradArgs &g, const float *dw, const int32_t *count,
                                  const int32_t *tokens, const float *dloss, void *dlogits,
                                  int odt, size_t ldd, cudaStream_t stream) {
  RouteBackArgs a;
  a.g = g;
  a.lanes = team_lanes(g.r.n_expert);
  a.vec = g.r.n_expert % 8 == 0 && vec_rows(g.logits, g.dt, g.ld);
  a.vec_out = g.r.n_expert % 8 == 0 && vec_rows(dlogits, odt, ldd);
  a.dw = dw;
  a.count = count;
  a.tokens = tokens;
  a.dloss = dloss;
  a.dlogits = dlogits;
  a.odt = odt;
  a.ldd = ldd;
  const uint64_t groups = ((uint64_t)g.t.T + 32 / a.lanes - 1) / (32 / a.lanes);
  const uint64_t warps = (uint64_t)fp8_ctas() * 4 * kWarps;
  a.run = (uint32_t)((groups + warps - 1) / warps);
  const unsigned grid = (unsigned)((groups + (uint64_t)a.run * kWarps - 1) / ((uint64_t)a.run * kWarps));
  if (g.dt == MOE_DT_F32) return route_backward_t<MOE_DT_F32>(a, grid, stream);
  if (g.dt == MOE_DT_BF16) return route_backward_t<MOE_DT_BF16>(a, grid, stream);
  return route_backward_t<MOE_DT_F16>(a, grid, stream);
}

cudaError_t launch_combine_backward(const void *dy, int ydt, size_t ldy, const void *o, int dt,
                                    size_t ldo, uint32_t R, const float *w, const int32_t *pos,
                                    uint32_t T, uint32_t k, uint32_t d, float *dw, void *dout,
                                    size_t ldd, cudaStream_t stream) {
  const CombineBackArgs a{dy, ldy, o, ldo, R, w, pos, T, k, d, dw, dout, ldd};
  if (dt == MOE_DT_F32) return combine_backward_from<MOE_DT_F32>(ydt, a, stream);
  if (dt == MOE_DT_BF16) return combine_backward_from<MOE_DT_BF16>(ydt, a, stream);
  return combine_backward_from<MOE_DT_F16>(ydt, a, stream);
}

}  // namespace moe
