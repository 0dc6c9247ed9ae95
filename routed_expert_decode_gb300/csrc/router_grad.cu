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
// CTAs an SM of the logits' gradient by a lane's chunks of experts, all of a grid at a time
// (before the tests for tiny scores, 65536 x 256 bf16: 33 us, 34 with 4; 32768 x 512: 29, and 37
// with a grid of 3)
constexpr int back_ctas(int nc) { return nc == 1 ? 3 : nc == 2 ? 2 : 1; }
constexpr int kThreads = kWarps * 32;
constexpr uint32_t kAll = 0xffffffffu;

// WIDE: teams of 32 lanes, known when compiling; else of a power of two below
template <bool WIDE>
struct Team {
  uint32_t few;  // a narrow team's lanes
  int l, t;      // lane within the team, team within the warp
  __device__ __forceinline__ explicit Team(uint32_t lanes) : few(lanes) {
    const int lane = threadIdx.x & 31;
    l = WIDE ? lane : lane & (int)(lanes - 1);
    t = WIDE ? 0 : lane / (int)lanes;
  }
  __device__ __forceinline__ uint32_t lanes() const { return WIDE ? 32 : few; }
  __device__ __forceinline__ uint32_t per_warp() const { return WIDE ? 1 : 32 / few; }
  __device__ __forceinline__ uint32_t expert(int c) const { return (c * lanes() + l) * 8; }
  __device__ __forceinline__ float sum(float v) const {
    if (WIDE) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    } else {
      for (uint32_t o = few >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    }
    return v;
  }
  __device__ __forceinline__ float max(float v) const {
    if (WIDE) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    } else {
      for (uint32_t o = few >> 1; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    }
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

// One token's logits; lanes and elements without an expert hold -inf, whose score is 0.
template <int DT, int NC>
struct Row {
  Raw8<DT> raw[NC];
  template <typename Team>
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
  __device__ __forceinline__ void to(float2 (&l)[NC][4]) const {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float f[8];
      raw[c].to(f);
#pragma unroll
      for (int i = 0; i < 4; ++i) l[c][i] = make_float2(f[2 * i], f[2 * i + 1]);
    }
  }
};

// arithmetic on two fp32 values an instruction
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// e^(-x/2) for |x| up to 180 (0 at 180): 2^(-x/2 log2 e) by the special function unit, with
// the roundings of the product and of log2 e made good, as those of an argument of 80
// would be 40 ulp.  Within 2 ulp.
__device__ __forceinline__ float2 exp_of_minus_half(float2 x) {
  constexpr float kHi = 1.4426950216293335f, kLo = 1.9259629911266175e-8f;  // log2 e
  constexpr float kLn2 = 0.6931471805599453f;
  const float2 t = mul2(x, both(0.5f * kHi));
  // half of what is missing from the exponent
  const float2 rest = fma2(x, both(-0.5f * kLo), fma2(x, both(-0.5f * kHi), t));
  float2 e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(-t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(-t.y));
  return fma2(mul2(e, both(kLn2)), rest, e);
}
// e^-x for |x| up to 110 (0 at 110, infinite below -88.7): a square, so that a subnormal
// result is not flushed.  Within 4 ulp.
__device__ __forceinline__ float2 exp_of_minus(float2 x) {
  const float2 h = exp_of_minus_half(x);
  return mul2(h, h);
}
// 1 / x within an ulp; 0 for x above 2^126
__device__ __forceinline__ float2 rcp2(float2 x) {
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(x.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(x.y));
  return r;
}

// sqrt(log(1 + e^l)), and its slope's d log / dl = sigmoid(l) / (2 log(1 + e^l)), of two l.
// With e = e^-|l|, log(1 + e) = e q, where q = 2/(2+e) (1 + z/3 + z^2/5 + ...) of z =
// (e/(2+e))^2 <= 1/9 is the series of 2 artanh(e/(2+e)), cut where 1.5e-8 is left.  Below 0 the
// root is e^(-|l|/2) sqrt(q) and the slope 1 / (2 (1+e) q), so that neither underflows before
// the root itself does; from 0 on they are of l + e q.  Both within 6 ulp.
template <bool SLOPE>
__device__ __forceinline__ float2 softplus_root(float2 l, float2 &slope) {
  const float2 h = exp_of_minus_half(
      make_float2(fminf(fabsf(l.x), 180.0f), fminf(fabsf(l.y), 180.0f)));
  const float2 e = mul2(h, h), r = rcp2(add2(e, both(2.0f)));
  const float2 t = mul2(e, r), z = mul2(t, t);
  float2 q = fma2(z, both(1.0f / 13), both(1.0f / 11));
  q = fma2(q, z, both(1.0f / 9));
  q = fma2(q, z, both(1.0f / 7));
  q = fma2(q, z, both(1.0f / 5));
  q = fma2(q, z, both(1.0f / 3));
  q = mul2(fma2(q, z, both(1.0f)), add2(r, r));
  const bool ux = l.x >= 0.0f, uy = l.y >= 0.0f;  // NaN: as -inf
  const float2 up = fma2(e, q, make_float2(fminf(l.x, FLT_MAX), fminf(l.y, FLT_MAX)));
  const float2 v = make_float2(ux ? up.x : q.x, uy ? up.y : q.y);
  float2 root;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(root.x) : "f"(v.x));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(root.y) : "f"(v.y));
  if (SLOPE)
    slope = mul2(mul2(mul2(rcp2(add2(e, both(1.0f))), both(0.5f)), root), root);
  return mul2(mul2(v, root), make_float2(ux ? 1.0f : h.x, uy ? 1.0f : h.y));
}

// l -> scores p (softmax: whose sum is 1), in place; slope = d log p / dl, softmax's
// without its sum's part.  A NaN counts as -inf, +inf as the largest finite value.
// Returns the sum of p (without SLOPE, sigmoid's p and sum are four times those); top and norm:
// softmax's maximum of l and the factor of e^(l - top).
template <int NC, bool SLOPE, typename Team>
__device__ __forceinline__ float scores(uint32_t fn, const Team &tm, float2 (&l)[NC][4],
                                        float2 (&slope)[NC][4], float &top, float &norm) {
  float2 s = both(0.0f);
  if (fn == MOE_SCORE_SOFTMAX) {
    float m = -FLT_MAX;  // of a row of -inf: every term is 0
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 &v = l[c][i];
        v.x = fminf(fmaxf(v.x, -INFINITY), FLT_MAX);
        v.y = fminf(fmaxf(v.y, -INFINITY), FLT_MAX);
        m = fmaxf(m, fmaxf(v.x, v.y));
      }
    m = tm.max(m);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 &v = l[c][i];
        v = exp_of_minus(make_float2(fminf(m - v.x, 110.0f), fminf(m - v.y, 110.0f)));
        s = add2(s, v);
        if (SLOPE) slope[c][i] = both(1.0f);
      }
    const float sum = tm.sum(s.x + s.y);
    const float r = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
    top = m;
    norm = r;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) l[c][i] = mul2(l[c][i], both(r));
    return sum > 0.0f ? 1.0f : 0.0f;
  }
  if (fn == MOE_SCORE_SIGMOID) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = l[c][i];
        if (SLOPE) {
          // of e = e^-|l|: 1/(1+e) is the larger of sigmoid(l) and sigmoid(-l), e/(1+e) the other
          const float2 e = exp_of_minus(
              make_float2(fminf(fabsf(v.x), 110.0f), fminf(fabsf(v.y), 110.0f)));
          const float2 big = rcp2(add2(e, both(1.0f))), small = mul2(e, big);
          const bool ux = v.x >= 0.0f, uy = v.y >= 0.0f;  // NaN: as -inf
          l[c][i] = make_float2(ux ? big.x : small.x, uy ? big.y : small.y);
          slope[c][i] = make_float2(ux ? small.x : big.x, uy ? small.y : big.y);
        } else {
          const float2 e = exp_of_minus(make_float2(fminf(fmaxf(v.x, -110.0f), 110.0f),
                                                    fminf(fmaxf(v.y, -110.0f), 110.0f)));
          // four times p, which shares do not see: rcp2 is not 0 before e is infinite
          l[c][i] = rcp2(fma2(e, both(0.25f), both(0.25f)));
        }
        s = add2(s, l[c][i]);
      }
    return tm.sum(s.x + s.y);
  }
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 &v = l[c][i];
      v = softplus_root<SLOPE>(v, slope[c][i]);
      s = add2(s, v);
    }
  return tm.sum(s.x + s.y);
}

// Scores that add up to less than this are taken 2^64 times, which is exact: the reciprocal
// of their sum may be infinite otherwise (a sum below 2^-128), and products with them lose
// bits as subnormal numbers.
constexpr float kTinySum = 0x1p-64f, kTinyScale = 0x1p64f;
// The router's sigmoid is 1 / (1 + e^-l), and 0 where e^-l is infinite: at logits below
// kLeastLogit, whose p are below kLeastScore.  They count as 0 here where it matters: picks, and
// tokens whose scores are tiny in all.  (sqrt(softplus) goes on as e^(l/2) down to -174.7; the
// router's has few bits below -87 and is 0 below -103.97.)
constexpr float kLeastLogit = -88.72283f, kLeastScore = 0x1.00004p-128f;
__device__ __forceinline__ bool tiny_sum(float sum) { return sum > 0.0f && sum < kTinySum; }

// p of one logit; softmax: e^(l - top), and 0 for -inf whatever top is
__device__ __forceinline__ float score_of(uint32_t fn, float l, float top) {
  if (fn == MOE_SCORE_SOFTMAX) return exp_of_minus(both(fminf(top - l, 110.0f))).x;
  if (fn == MOE_SCORE_SIGMOID) {
    const float e = exp_of_minus(both(fminf(fabsf(l), 110.0f))).x;
    const float big = rcp2(both(1.0f + e)).x;
    return l >= 0.0f ? big : l < kLeastLogit ? 0.0f : e * big;
  }
  float2 none;
  return softplus_root<false>(both(l), none).x;
}

// ---------------------------------------------------------------- sequences
__device__ __forceinline__ int seq_at(const moe_tokens &t, uint32_t s) {
  return t.seq ? min(max(t.seq[s], 0), (int)t.T) : s == 0 ? 0 : (int)t.T;
}
// The first sequence that ends behind token x (S: none), by a whole warp: as many as end at
// or before it, counted 32 at a time for few sequences.
__device__ __forceinline__ uint32_t seq_of(const moe_tokens &t, int x) {
  uint32_t lo = 0, hi = t.S;
  if (hi <= 128) {
#pragma unroll
    for (uint32_t i = 0; i < 128; i += 32) {
      const uint32_t s = i + (threadIdx.x & 31);
      if (i < hi) lo += __popc(__ballot_sync(kAll, s < hi && seq_at(t, min(s, hi - 1) + 1) <= x));
    }
    return lo;
  }
  while (lo < hi) {
    const uint32_t mid = (lo + hi) / 2;
    if (seq_at(t, mid + 1) > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// the first sequence from s on that ends behind token x (S: none), by a thread for itself
__device__ __forceinline__ uint32_t seq_from(const moe_tokens &t, uint32_t s, int x) {
  uint32_t lo = s, hi = t.S;
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
// an SM, by a lane's chunks of experts (65536 x 256 bf16, 16 sequences: 24 us, 26 with 2 or 4)
constexpr int sum_ctas(int nc) { return nc == 1 ? 3 : 2; }
constexpr uint32_t kSumPasses = 4;  // tokens of a team, at least
constexpr uint32_t kJoinRun = 32;   // experts of a joining CTA
constexpr uint32_t kAloneSeqs = 4;  // sequences of a call that one CTA finishes, at most

struct BalanceArgs {
  RouterGradArgs g;
  uint32_t lanes, per;
  bool vec;
  int32_t *count, *tokens;
  float *prob, *loss;
  float *part;         // [CTAs][2][E] sums of shares
  int32_t *part_count;  // [CTAs][2][E] picks
  int32_t *part_n;      // [CTAs][2] counting tokens
  float *seq_loss;     // [S][chunks]: terms of the loss by runs of experts
  uint32_t chunks;     // runs of kJoinRun experts
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

// a sequence's factor of the loss: E / (k n)
__device__ __forceinline__ float seq_factor(const BalanceArgs &a, int n) {
  return n > 0 ? __fdiv_rn((float)a.g.r.n_expert, (float)a.g.r.top_k * (float)n) : 0.0f;
}
// one expert's outputs from its sums; returns its term of the loss up to the factor
__device__ __forceinline__ float finish_expert(const BalanceArgs &a, uint32_t s, uint32_t e, int n,
                                               int picks, float shares) {
  const float p = n > 0 ? __fdiv_rn(shares, (float)n) : 0.0f;
  a.count[(size_t)s * a.g.r.n_expert + e] = picks;
  a.prob[(size_t)s * a.g.r.n_expert + e] = p;
  return (float)picks * p;
}

// the loss from the sequences' terms, by one block
template <int THREADS>
__device__ __forceinline__ void finish_loss(const BalanceArgs &a, float *red) {
  float v = 0.0f;
  for (uint32_t i = threadIdx.x; i < a.g.t.S * a.chunks; i += THREADS) v += __ldcg(a.seq_loss + i);
  v = block_sum<THREADS>(v, red);
  if (threadIdx.x == 0) a.loss[0] = v * __fdiv_rn(a.g.coef, (float)a.g.t.S);
}

template <int DT, int NC, bool WIDE>
__global__ void __launch_bounds__(kThreads, sum_ctas(NC)) k_balance(const BalanceArgs a) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ __align__(16) uint8_t bsm[];
  const uint32_t E = a.g.r.n_expert, k = a.g.r.top_k;
  const Team<WIDE> tm(a.lanes);
  const uint32_t width = NC * tm.lanes() * 8;
  float *red = (float *)bsm;                     // [kWarps][width]
  int *cnt = (int *)(red + kWarps * width);      // [width]
  __shared__ float sums[32];
  __shared__ int live_n;
  const int tid = threadIdx.x, warp = tid >> 5;
  const bool alone = gridDim.x == 1 && a.g.t.S <= kAloneSeqs;
  const int t0 = (int)min(a.g.t.T, blockIdx.x * a.per);
  const int t1 = (int)min((uint64_t)a.g.t.T, (uint64_t)t0 + a.per);
  constexpr int U = NC == 1 ? 2 : 1;  // tokens of a team at a time, the next on their way
  const int step = kWarps * (int)tm.per_warp();
  for (uint32_t s = alone ? 0 : seq_of(a.g.t, t0), after; s < a.g.t.S; s = after) {
    after = s + 1;
    const int s0 = seq_at(a.g.t, s), s1 = seq_at(a.g.t, s + 1);
    if (!alone && s0 >= t1) break;
    const int lo = max(s0, t0), hi = min(s1, t1);
    if (!alone && lo >= hi) {  // no tokens: to the next that has some
      after = max(after, seq_of(a.g.t, lo));
      continue;
    }
    for (uint32_t e = tid; e < width; e += kThreads) cnt[e] = 0;
    if (tid == 0) live_n = 0;
    __syncthreads();
    // the picks of this thread's first token, on the way during the sum of the shares
    constexpr uint32_t kAhead = 8;
    const int first = lo + tid;
    int32_t ahead[kAhead];
    const bool counting = first < hi && (!a.g.t.live || a.g.t.live[first]);
#pragma unroll
    for (uint32_t j = 0; j < kAhead; ++j)
      ahead[j] = counting && j < k ? a.g.idx[(size_t)first * k + j] : -1;
    // ---- shares
    float2 acc[NC][4];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[c][i] = both(0.0f);
    Row<DT, NC> row[U], next[U];
    bool on[U], next_on[U];
    auto fetch = [&](Row<DT, NC>(&r)[U], bool(&o)[U], int base) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = base + u * step + tm.t;
        o[u] = t < hi && (!a.g.t.live || a.g.t.live[t]);
        r[u].load(a.g.logits, a.g.ld, (uint32_t)t, E, tm, a.vec, o[u]);
      }
    };
    fetch(row, on, lo + warp * (int)tm.per_warp());
    for (int base = lo + warp * (int)tm.per_warp(); base < hi; base += U * step) {
      fetch(next, next_on, base + U * step);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float2 l[NC][4];
        row[u].to(l);
        float top, norm;
        const float sum = scores<NC, false>(a.g.r.score, tm, l, l, top, norm);
        const float inv = on[u] && sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[c][i] = fma2(l[c][i], both(inv), acc[c][i]);
        row[u] = next[u];
        on[u] = next_on[u];
      }
    }
    // ---- picks, a thread a token
    int mine = counting;
#pragma unroll
    for (uint32_t j = 0; j < kAhead; ++j)
      if ((uint32_t)ahead[j] < E) atomicAdd(&cnt[ahead[j]], 1);
    for (int t = first; t < hi; t += kThreads) {
      uint32_t j = 0;
      if (t == first) {
        if (!counting) continue;
        j = kAhead;
      } else {
        if (a.g.t.live && !a.g.t.live[t]) continue;
        ++mine;
      }
      for (; j < k; ++j) {
        const uint32_t e = (uint32_t)a.g.idx[(size_t)t * k + j];
        if (e < E) atomicAdd(&cnt[e], 1);
      }
    }
    mine = __reduce_add_sync(kAll, mine);
    if (mine && (tid & 31) == 0) atomicAdd(&live_n, mine);
    // ---- the warps' shares in order
    for (uint32_t o = tm.lanes(); o < 32; o <<= 1)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[c][i].x += __shfl_xor_sync(kAll, acc[c][i].x, o);
          acc[c][i].y += __shfl_xor_sync(kAll, acc[c][i].y, o);
        }
    if (tm.t == 0)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *(float2 *)(red + warp * width + tm.expert(c) + 2 * i) = acc[c][i];
    __syncthreads();
    auto shares = [&](uint32_t e) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += red[w * width + e];
      return v;
    };
    if (s0 >= t0 && s1 <= t1) {
      const int n = live_n;
      float loss = 0.0f;
      for (uint32_t e = tid; e < E; e += kThreads)
        loss += finish_expert(a, s, e, n, cnt[e], shares(e));
      loss = block_sum<kThreads>(loss, sums);
      if (tid == 0) a.tokens[s] = n;
      if ((uint32_t)tid < a.chunks)
        a.seq_loss[s * a.chunks + tid] = tid == 0 ? loss * seq_factor(a, n) : 0.0f;
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

// The sequences that no CTA had to itself, empty ones, and the loss.  A CTA joins a run of
// 32 experts of a sequence, a warp every 16th of its parts; the last one adds up the loss.
__global__ void __launch_bounds__(kJoinThreads) k_balance_join(const BalanceArgs a) {
  pdl_trigger();
  pdl_wait();
  constexpr int kGroups = kJoinThreads / (int)kJoinRun;
  __shared__ float sums[32];
  __shared__ float share_g[kGroups][kJoinRun];
  __shared__ int count_g[kGroups][kJoinRun];
  __shared__ int live_n;
  __shared__ bool last;
  const uint32_t E = a.g.r.n_expert;
  const int tid = threadIdx.x, g = tid / (int)kJoinRun, l = tid % (int)kJoinRun;
  const uint32_t items = a.g.t.S * a.chunks;
  for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
    const uint32_t s = item / a.chunks, chunk = item - s * a.chunks, e = chunk * kJoinRun + l;
    const int s0 = seq_at(a.g.t, s), s1 = seq_at(a.g.t, s + 1);
    const uint32_t c0 = (uint32_t)s0 / a.per, c1 = s0 < s1 ? (uint32_t)(s1 - 1) / a.per : c0;
    if (s0 < s1 && c0 == c1) continue;  // its CTA has written it
    // the sequence begins among the tokens of c0
    auto slot = [&](uint32_t c) { return (size_t)c * 2 + ((uint32_t)s0 >= c * a.per); };
    __syncthreads();
    if (tid == 0) live_n = 0;
    __syncthreads();
    int n = 0, picks = 0;
    float v = 0.0f;
    if (s0 < s1) {
      for (uint32_t c = c0 + tid; c <= c1; c += kJoinThreads) n += __ldcg(a.part_n + slot(c));
      if (n) atomicAdd(&live_n, n);
      if (e < E)
#pragma unroll 8
        for (uint32_t c = c0 + g; c <= c1; c += kGroups) {
          v += __ldcg(a.part + slot(c) * E + e);
          picks += __ldcg(a.part_count + slot(c) * E + e);
        }
    }
    share_g[g][l] = v;
    count_g[g][l] = picks;
    __syncthreads();
    if (g == 0) {
      n = live_n;
      v = 0.0f;
      picks = 0;
#pragma unroll
      for (int q = 0; q < kGroups; ++q) {
        v += share_g[q][l];
        picks += count_g[q][l];
      }
      float loss = e < E ? finish_expert(a, s, e, n, picks, v) : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) loss += __shfl_xor_sync(kAll, loss, o);
      if (l == 0) {
        a.seq_loss[item] = loss * seq_factor(a, n);
        if (chunk == 0) a.tokens[s] = n;
      }
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
  uint32_t lanes, run;  // of a team; tokens of a warp
  uint32_t slots;       // lanes for a token's picks, a power of two
  bool vec, vec_out;
  const float *dw;
  const int32_t *count, *tokens;
  const float *dloss;
  void *dlogits;
  int odt;
  size_t ldd;
};

template <int OT, int NC, typename Team>
__device__ __forceinline__ void store_row(const RouteBackArgs &a, uint32_t t, const Team &tm,
                                          bool vec, const float2 (&d2)[NC][4]) {
  typename Elem<OT>::T *row = (typename Elem<OT>::T *)a.dlogits + (size_t)t * a.ldd;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const uint32_t e = tm.expert(c);
    const float d[8] = {d2[c][0].x, d2[c][0].y, d2[c][1].x, d2[c][1].y,
                        d2[c][2].x, d2[c][2].y, d2[c][3].x, d2[c][3].y};
    if (vec) {
      if (e < a.g.r.n_expert) store8<OT>(row + e, d);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < a.g.r.n_expert) row[e + i] = Elem<OT>::from(d[i]);
    }
  }
}

// A warp takes `run` consecutive tokens, in batches.  First the picks of a whole batch, a lane a
// slot (four tokens of up to 8 slots): their logits are read and scored by themselves, and
// their part of the gradient goes to rows of zeros in shared memory.  Then the tokens, each
// by its team, the next one's logits on their way: scores, the loss's part (whose
// coefficients stay in registers from token to token), the picks' part from shared memory.
// FAST: sigmoid, whole chunks of 8 in and out, the gradient of the logits' type, known when
// compiling.
// 65536 x 256 bf16, top 8, with the loss: 34.1 to 34.5 us, of which scores and stores alone are
// some 20 and the tests for tiny scores 0.5.  Without those 33.0; 35.0 without FAST, and then
// 37.7 with longer runs for fewer CTAs, 39.1 with the picks token by token, from p laid out in
// shared memory.  Neither issue (0.57) nor HBM (0.13) is full: a token's sums wait on each other.
template <int DT, int NC, bool WIDE, bool FAST>
__global__ void __launch_bounds__(kThreads, back_ctas(NC))
    k_route_backward(const RouteBackArgs a) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ __align__(16) uint8_t rsm[];
  const uint32_t E = a.g.r.n_expert, k = a.g.r.top_k, T = a.g.t.T;
  const uint32_t fn = FAST ? MOE_SCORE_SIGMOID : a.g.r.score;
  const int odt = FAST ? DT : a.odt;
  const bool vec = FAST || a.vec, vec_out = FAST || a.vec_out;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Team<WIDE> tm(a.lanes);
  const uint32_t width = NC * tm.lanes() * 8, nt = tm.per_warp();
  const uint32_t slots = a.slots, nb = 32 / slots;     // lanes of a token's picks, tokens
  const uint32_t batch = nb > nt ? nb : nt;            // tokens of a batch
  float *vbuf = (float *)rsm + (size_t)warp * batch * (width + 4);  // [batch][width] zeros
  float *stat = vbuf + batch * width;                   // [batch][4] top and sum of the picks
  const uint64_t first = ((uint64_t)blockIdx.x * kWarps + warp) * a.run;
  if (first >= T) return;
  const uint32_t t0 = (uint32_t)first, t1 = (uint32_t)min((uint64_t)T, first + a.run);
  const bool softmax = fn == MOE_SCORE_SOFTMAX;
  for (uint32_t i = lane * 4; i < batch * (width + 4); i += 128)
    *(float4 *)(vbuf + i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  // factor of a sequence's loss gradient, up to 1 / n^2
  const float factor =
      a.count ? (a.dloss ? a.dloss[0] : 1.0f) *
                    __fdiv_rn(a.g.coef * (float)E, (float)a.g.t.S * (float)k)
              : 0.0f;
  uint32_t s = a.count ? seq_of(a.g.t, (int)t0) : 0;
  int s_begin = 0, s_end = 0;
  uint32_t have = 0xffffffffu;  // the sequence whose coefficients coef holds
  float2 coef[NC][4];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) coef[c][j] = both(0.0f);
  if (a.count && s < a.g.t.S) {
    s_begin = seq_at(a.g.t, s);
    s_end = seq_at(a.g.t, s + 1);
  }
  // ---- this lane's slot of a batch: pick (E: none) and dw two batches ahead, its logit one
  const uint32_t slot = (uint32_t)lane & (slots - 1), of = (uint32_t)lane / slots;
  auto pick_at = [&](uint32_t x, uint32_t &e, float &g) {
    const bool in = a.dw && slot < k && x < t1;
    e = in ? min((uint32_t)a.g.idx[(size_t)x * k + slot], E) : E;
    g = e < E ? a.dw[(size_t)x * k + slot] : 0.0f;
  };
  auto logit_at = [&](uint32_t x, uint32_t e) {
    using X = Elem<DT>;
    return e < E ? logit_value(X::to(((const typename X::T *)a.g.logits)[(size_t)x * a.g.ld + e]))
                 : -INFINITY;
  };
  auto group_sum = [&](float v) {
    for (uint32_t o = slots >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
  };
  // one lane's slot: its part of the gradient to row r
  auto picks = [&](uint32_t r, uint32_t e, float g, float l) {
    float top = 0.0f;
    if (softmax) {  // of the picks: the row's is not known yet
      top = e < E ? l : -FLT_MAX;
      for (uint32_t o = slots >> 1; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
      top = fmaxf(top, -FLT_MAX);
    }
    float p = e < E ? score_of(fn, l, top) : 0.0f;
    float dots = group_sum(p * g);
    float v = a.g.r.s * p * g;
    if (a.g.r.renorm) {
      float total = group_sum(p);
      if (__any_sync(kAll, tiny_sum(total))) {
        const float f = tiny_sum(total) ? kTinyScale : 1.0f;
        p *= f;
        total *= f;
        dots = group_sum(p * g);
      }
      const float inv = total > 0.0f ? __fdiv_rn(1.0f, total) : 0.0f;
      v = a.g.r.s * (p * inv) * (g - dots * inv);
    }
    if (softmax && slot == 0) {
      stat[4 * r] = top;
      stat[4 * r + 1] = dots;
    }
    // the lanes one after another where two of them have the same expert
    const uint32_t key = e < E ? r * 1024 + e : 0x80000000u + (uint32_t)lane;
    const uint32_t same = __match_any_sync(kAll, key);
    const uint32_t before = __popc(same & ((1u << lane) - 1u));
    for (uint32_t turn = 0; __any_sync(kAll, before >= turn); ++turn) {
      if (before == turn && e < E) vbuf[r * width + e] += v;
      __syncwarp();
    }
  };
  uint32_t e1, e2;
  float g1, g2, l1;
  pick_at(t0 + of, e1, g1);
  l1 = logit_at(t0 + of, e1);
  pick_at(t0 + batch + of, e2, g2);
  Row<DT, NC> next;
  bool next_live = true;
  auto fetch = [&](uint32_t x) {
    next.load(a.g.logits, a.g.ld, x, E, tm, vec, x < t1);
    if (a.count && a.g.t.live) next_live = x < t1 && a.g.t.live[x];
  };
  fetch(t0 + tm.t);
  __syncwarp();
  for (uint32_t b0 = t0; b0 < t1; b0 += batch) {
    if (a.dw) {
      picks(of, e1, g1, l1);
      for (uint32_t sub = nb; sub < batch; sub += nb) {  // teams of more tokens than that
        uint32_t e;
        float g;
        pick_at(b0 + sub + of, e, g);
        picks(sub + of, e, g, logit_at(b0 + sub + of, e));
      }
    }
    const uint32_t e0 = e1;
    e1 = e2;
    g1 = g2;
    l1 = logit_at(b0 + batch + of, e1);
    pick_at(b0 + 2 * batch + of, e2, g2);
    for (uint32_t i = 0; i < batch && b0 + i < t1; i += nt) {
      const uint32_t t = b0 + i + tm.t;
      const bool on = t < t1, live = next_live;
      float2 p[NC][4], slope[NC][4], d[NC][4];
      next.to(p);
      if (b0 + i + nt < t1) fetch(t + nt);
      float top = 0.0f, norm = 0.0f;
      float sum = scores<NC, true>(fn, tm, p, slope, top, norm);
      // ---- the loss's part
      bool counts = false;
      if (a.count && on) {
        if (s < a.g.t.S && s_end <= (int)t) {
          ++s;
          if (s < a.g.t.S && seq_at(a.g.t, s + 1) <= (int)t) s = seq_from(a.g.t, s + 1, (int)t);
          if (s < a.g.t.S) {
            s_begin = seq_at(a.g.t, s);
            s_end = seq_at(a.g.t, s + 1);
          }
        }
        counts = s < a.g.t.S && s_begin <= (int)t && live;
        if (counts && s != have) {
          const int32_t *cs = a.count + (size_t)s * E;
          const float n = (float)max(a.tokens[s], 1), f = __fdiv_rn(factor, n * n);
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t e = tm.expert(c) + 2 * j;
              coef[c][j] = make_float2(e < E ? f * (float)cs[e] : 0.0f,
                                       e + 1 < E ? f * (float)cs[e + 1] : 0.0f);
            }
          have = s;
        }
      }
      if (__any_sync(kAll, counts)) {
        auto weighted = [&]() {  // sum of coef p
          float2 dots = both(0.0f);
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) dots = fma2(coef[c][j], p[c][j], dots);
          return tm.sum(dots.x + dots.y);
        };
        float dot = weighted();
        if (__any_sync(kAll, tiny_sum(sum))) {
          const bool tiny = tiny_sum(sum);
          float2 some = both(0.0f);
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float2 &v = p[c][j];
              if (tiny)
                v = make_float2(v.x < kLeastScore ? 0.0f : v.x * kTinyScale,
                                v.y < kLeastScore ? 0.0f : v.y * kTinyScale);
              some = add2(some, v);
            }
          const float again = tm.sum(some.x + some.y);
          if (tiny) sum = again;
          dot = weighted();
        }
        const float inv = counts && sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
        dot *= inv;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            d[c][j] = mul2(mul2(p[c][j], both(inv)), add2(coef[c][j], both(-dot)));
      } else {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) d[c][j] = both(0.0f);
      }
      // ---- the picks' part
      if (a.dw) {
        const uint32_t r = i + tm.t;
        float f = 1.0f;
        if (softmax) {  // beside the row's largest logit; picks whose p is 0 weigh nothing
          f = exp_of_minus(both(fminf(fmaxf(top - stat[4 * r], 0.0f), 110.0f))).x * norm;
          if (a.g.r.renorm) f = f > 0.0f ? 1.0f : 0.0f;
        }
        if (softmax && !a.g.r.renorm) {  // every expert's p falls as a pick's rises
          const float fall = -a.g.r.s * (stat[4 * r + 1] * f);
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) d[c][j] = fma2(both(fall), p[c][j], d[c][j]);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float4 *b = (const float4 *)(vbuf + r * width + tm.expert(c));
          const float4 x = b[0], y = b[1];
          d[c][0] = fma2(both(f), make_float2(x.x, x.y), d[c][0]);
          d[c][1] = fma2(both(f), make_float2(x.z, x.w), d[c][1]);
          d[c][2] = fma2(both(f), make_float2(y.x, y.y), d[c][2]);
          d[c][3] = fma2(both(f), make_float2(y.z, y.w), d[c][3]);
        }
      }
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) d[c][j] = mul2(d[c][j], slope[c][j]);
      if (!on) continue;
      if (odt == MOE_DT_F32) store_row<MOE_DT_F32, NC>(a, t, tm, vec_out, d);
      else if (odt == MOE_DT_BF16) store_row<MOE_DT_BF16, NC>(a, t, tm, vec_out, d);
      else store_row<MOE_DT_F16, NC>(a, t, tm, vec_out, d);
    }
    if (!a.dw) continue;
    __syncwarp();
    if (batch == nb) {
      if (e0 < E) vbuf[of * width + e0] = 0.0f;
    } else {
      for (uint32_t i = lane * 4; i < batch * width; i += 128)
        *(float4 *)(vbuf + i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    __syncwarp();
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
// others.  DEEP: steps of 256 values whose loads go out together, before any store.
template <int DT, int YT, bool VEC, int DEEP>
__global__ void __launch_bounds__(kThreads) k_combine_backward(const CombineBackArgs a) {
  pdl_trigger();
  pdl_wait();
  using X = Elem<DT>;
  using Y = Elem<YT>;
  const int lane = threadIdx.x & 31;
  const uint32_t it = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (it < a.T * a.k) {
    const uint32_t t = it / a.k;
    const uint32_t r = (uint32_t)a.pos[it];
    if (r >= a.R) {
      if (a.dw && lane == 0) a.dw[it] = 0.0f;
      return;
    }
    const typename Y::T *y = (const typename Y::T *)a.dy + (size_t)t * a.ldy;
    const typename X::T *o = (const typename X::T *)a.o + (size_t)r * a.ldo;
    typename X::T *g = (typename X::T *)a.dout + (size_t)r * a.ldd;
    const float w = a.dout ? a.w[it] : 0.0f;
    float sum = 0.0f;
    for (uint32_t c0 = lane * 8; c0 < a.d; c0 += 256 * DEEP) {
      Raw8<DT> ro[DEEP];
      Raw8<YT> ry[DEEP];
#pragma unroll
      for (int u = 0; u < DEEP; ++u) {
        const uint32_t c = c0 + 256 * u;
        if (VEC) {
          if (c >= a.d) break;
          if (a.dw) ro[u].load(o + c);
          const uint4 *q = (const uint4 *)(y + c);
#pragma unroll
          for (int i = 0; i < (YT == MOE_DT_F32 ? 2 : 1); ++i) ry[u].v[i] = q[i];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (a.dw) ((typename X::T *)ro[u].v)[i] = c + i < a.d ? o[c + i] : X::from(0.0f);
            ((typename Y::T *)ry[u].v)[i] = c + i < a.d ? y[c + i] : Y::from(0.0f);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < DEEP; ++u) {
        const uint32_t c = c0 + 256 * u;
        if (c >= a.d) break;
        float fy[8], fo[8];
        ry[u].to(fy);
        if (a.dw) {
          ro[u].to(fo);
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
  if (a.lanes < 32) return launch_k(k_balance<DT, 1, false>, grid, kThreads, smem, stream, true, a);
  if (nc == 1) return launch_k(k_balance<DT, 1, true>, grid, kThreads, smem, stream, true, a);
  if (nc == 2) return launch_k(k_balance<DT, 2, true>, grid, kThreads, smem, stream, true, a);
  return launch_k(k_balance<DT, 4, true>, grid, kThreads, smem, stream, true, a);
}

template <int DT>
cudaError_t route_backward_t(const RouteBackArgs &a, unsigned grid, cudaStream_t stream) {
  const int nc = chunks_of(a.g.r.n_expert);
  const uint32_t width = nc * a.lanes * 8, nt = 32 / a.lanes, nb = 32 / a.slots;
  const size_t smem = (size_t)kWarps * (nb > nt ? nb : nt) * (width + 4) * 4;
  auto run = [&](auto kern, std::atomic<bool> *done) {
    const cudaError_t e = allow_smem(kern, done);
    return e != cudaSuccess ? e : launch_k(kern, grid, kThreads, smem, stream, true, a);
  };
  static std::atomic<bool> done[6][kMaxDevices];
  const bool fast = a.g.r.score == MOE_SCORE_SIGMOID && a.vec && a.vec_out && a.odt == DT;
  if (a.lanes < 32) return run(k_route_backward<DT, 1, false, false>, done[0]);
  if (nc == 1 && fast) return run(k_route_backward<DT, 1, true, true>, done[1]);
  if (nc == 1) return run(k_route_backward<DT, 1, true, false>, done[2]);
  if (nc == 2 && fast) return run(k_route_backward<DT, 2, true, true>, done[3]);
  if (nc == 2) return run(k_route_backward<DT, 2, true, false>, done[4]);
  return run(k_route_backward<DT, 4, true, false>, done[5]);
}

template <int DT, int YT>
cudaError_t combine_backward_t(const CombineBackArgs &a, cudaStream_t stream) {
  // below 2^27, as the host checked
  const unsigned grid = (unsigned)(((uint64_t)a.T * a.k + kWarps - 1) / kWarps);
  const bool vec = a.d % 8 == 0 && vec_rows(a.dy, YT, a.ldy) && (!a.dw || vec_rows(a.o, DT, a.ldo)) &&
                   (!a.dout || vec_rows(a.dout, DT, a.ldd));
  // four steps at least: 4096 tokens' 8 rows of 6144 bf16 130 us, 139 step by step; rows of 768
  // 16.4 and 15.7, as then more warps fit.  Two steps of fp32 rows of 512 9.3, one 11.5.
  auto kern = !vec        ? k_combine_backward<DT, YT, false, 1>
              : a.d > 768 ? k_combine_backward<DT, YT, true, 4>
                          : k_combine_backward<DT, YT, true, DT == MOE_DT_F32 ? 2 : 1>;
  return launch_k(kern, grid, kThreads, 0, stream, true, a);
}

template <int DT>
cudaError_t combine_backward_from(int ydt, const CombineBackArgs &a, cudaStream_t stream) {
  if (ydt == MOE_DT_F32) return combine_backward_t<DT, MOE_DT_F32>(a, stream);
  if (ydt == MOE_DT_BF16) return combine_backward_t<DT, MOE_DT_BF16>(a, stream);
  return combine_backward_t<DT, MOE_DT_F16>(a, stream);
}

uint32_t balance_ctas(uint32_t T, uint32_t E) {
  const uint32_t least = kWarps * (32 / team_lanes(E)) * kSumPasses;  // tokens of a CTA
  const uint32_t n = (T + least - 1) / least;
  const uint32_t most = (uint32_t)(sum_ctas(chunks_of(E)) * fp8_ctas());
  return n < 1 ? 1 : n < most ? n : most;
}

}  // namespace

size_t balance_ws(const moe_router &r, uint32_t T, uint32_t S) {
  const size_t n = balance_ctas(T, r.n_expert), chunks = (r.n_expert + kJoinRun - 1) / kJoinRun;
  return MOE_WS_FIXED_BYTES + 4 * (n * 2 * (2 * (size_t)r.n_expert + 1) + S * chunks);
}

cudaError_t launch_balance(const RouterGradArgs &g, int32_t *count, int32_t *tokens, float *prob,
                           float *loss, void *ws, cudaStream_t stream) {
  BalanceArgs a;
  a.g = g;
  const uint32_t E = g.r.n_expert, n = balance_ctas(g.t.T, E);
  a.lanes = team_lanes(E);
  a.chunks = (E + kJoinRun - 1) / kJoinRun;
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
  if (e != cudaSuccess || (n == 1 && g.t.S <= kAloneSeqs)) return e;
  const uint32_t most = 4 * (uint32_t)fp8_ctas(), items = g.t.S * a.chunks;
  return launch_k(k_balance_join, items < most ? items : most, kJoinThreads, 0, stream, true, a);
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
  a.slots = 8;  // four tokens a batch: its rows of zeros are that many
  while (a.slots < g.r.top_k) a.slots *= 2;
  // As many warps as run at a time, with equal runs: whole batches each would leave every tenth
  // CTA out (65536 tokens: 410 of 456; 37.7 us in place of 35.0).
  const uint32_t nt = 32 / a.lanes;
  const uint64_t groups = ((uint64_t)g.t.T + nt - 1) / nt;  // of a team's tokens
  const uint64_t warps = (uint64_t)fp8_ctas() * back_ctas(chunks_of(g.r.n_expert)) * kWarps;
  a.run = (uint32_t)((groups + warps - 1) / warps) * nt;
  const unsigned grid =
      (unsigned)(((uint64_t)g.t.T + (uint64_t)a.run * kWarps - 1) / ((uint64_t)a.run * kWarps));
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
