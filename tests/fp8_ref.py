"""64-bit reference of the block-scaled fp8 operators (numpy), and the error bounds
their fp32 kernels are held to.  Shares no code with the library."""
import numpy as np

BLOCK = 128
U32 = 2.0 ** -24  # unit roundoff of fp32
MAX32 = float(np.finfo(np.float32).max)


def nb(n):
    return -(-n // BLOCK)


# ---------------------------------------------------------------- e4m3
def e4m3_values():
    """The 256 values of e4m3 (fn: no infinities; codes 0x7F and 0xFF are NaN)."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        a = m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        v[c] = np.nan if (e, m) == (15, 7) else (-a if s else a)
    return v


VALUES = e4m3_values()


def e4m3_encode(v):
    """Nearest e4m3 code of float64 values, ties to the even code, saturating; NaN -> 0x7F."""
    v = np.asarray(v, np.float64)
    pos = VALUES[:127]  # 0 .. 448 ascending
    a = np.abs(v)
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= 448.0, 126, code)
    code = code | np.where(np.signbit(v), 0x80, 0)
    return np.where(np.isnan(v), 0x7F, code).astype(np.uint8)


def quantize(x):
    """(codes, scales) of float32 rows by the definition: every operation of it is a
    single fp32 operation, so this is exact."""
    x = np.asarray(x, np.float32)
    T, d = x.shape
    pad = np.zeros((T, nb(d) * BLOCK), np.float32)
    pad[:, :d] = x
    b = pad.reshape(T, nb(d), BLOCK)
    a = np.fmax.reduce(np.abs(b), axis=2)  # a NaN does not enter
    a = np.fmax(a, np.float32(2.0 ** -100)).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        v = (b * (np.float32(448.0) / a)[:, :, None]).astype(np.float32)
    q = e4m3_encode(v).reshape(T, -1)[:, :d]
    nan = np.isnan(v).reshape(T, -1)[:, :d]
    return q, (a / np.float32(448.0)).astype(np.float32), nan


def dequantize(q, scale):
    n = q.shape[-1]
    return VALUES[q] * np.repeat(scale.astype(np.float64), BLOCK, axis=-1)[..., :n]


def weight(q, scale):
    """One expert's weights [N][K] in 64 bits."""
    N, K = q.shape
    s = np.repeat(np.repeat(scale.astype(np.float64), BLOCK, 0)[:N], BLOCK, 1)[:, :K]
    return VALUES[q] * s


def product(x, w):
    """x w^T in 64 bits and the elementwise bound of its fp32 evaluation.  A block's
    128 products are exact in fp32 and added in some order, each addition off by at
    most one fp32 ulp (a truncating adder; half that if it rounds); then a scale
    product, its use and the sum over the blocks, one rounding each."""
    ref = x @ w.T
    mag = np.abs(x) @ np.abs(w).T
    return ref, mag * (2 * U32 * BLOCK + U32 * (nb(x.shape[1]) + 4))


def swiglu(g, eg, u, eu):
    """h = g / (1 + e^-g) * u and its bound: the bounds of g and u carried through
    (|silu'| <= 1.1), and the roundings of e^-g (2 + 1.16|g| ulp of CUDA's fast
    exponential), the division (2 ulp) and three more operations."""
    with np.errstate(over="ignore"):
        s = g / (1.0 + np.exp(-g))
    h = s * u
    rel = 2 * U32 * (2 + 1.2 * np.abs(g) + 2 + 3)
    e = 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu + np.abs(h) * rel
    return h, e


# ---------------------------------------------------------------- router
def score(l, fn):
    """p in 64 bits: fn 0 sigmoid, 1 sqrt(softplus), 2 softmax.  NaN counts as
    -inf, +inf as the largest finite float32."""
    l = np.where(np.isnan(l), -np.inf, np.minimum(l.astype(np.float64), MAX32))
    with np.errstate(over="ignore", invalid="ignore"):
        if fn == 0:
            return l, 1.0 / (1.0 + np.exp(-l))
        if fn == 1:
            return l, np.sqrt(np.maximum(l, 0) + np.log1p(np.exp(-np.abs(l))))
        m = l.max(1, keepdims=True)
        e = np.where(l == -np.inf, 0.0, np.where(l == m, 1.0, np.exp(l - m)))
        s = e.sum(1, keepdims=True)
        return l, np.where(s > 0, e / np.where(s > 0, s, 1.0), 0.0)


def route(logits, bias, k, n_group, topk_group, fn, top2, renorm, s):
    """(idx, w, gap): picks and weights in 64 bits; gap[t] is the smallest difference
    between two selection values that token t's result rests on (the kept groups
    against the best dropped one, each pick against the next candidate).  Equal
    values (ties, resolved by index) do not count."""
    T, E = logits.shape
    l, p = score(logits, fn)
    by_logit = fn == 2 and bias is None and not top2
    c = l if by_logit else p
    if bias is not None:
        c = c + bias.astype(np.float64)
        c = np.where(np.isnan(c), -np.inf, c)
    gs = E // n_group
    idx = np.empty((T, k), np.int32)
    gap = np.full(T, np.inf)

    def note(t, a, b):
        if a != b and np.isfinite(a) and np.isfinite(b):
            gap[t] = min(gap[t], abs(a - b))

    for t in range(T):
        cand = list(range(E))
        if topk_group < n_group:
            sc = []
            for g in range(n_group):
                v = sorted(c[t, g * gs:(g + 1) * gs], reverse=True)
                sc.append(v[0] + v[1] if top2 and gs > 1 else v[0])
            order = sorted(range(n_group), key=lambda g: (-sc[g], g))
            note(t, sc[order[topk_group - 1]], sc[order[topk_group]])
            kept = set(order[:topk_group])
            cand = [e for e in cand if e // gs in kept]
        cand.sort(key=lambda e: (-c[t, e], e))
        idx[t] = cand[:k]
        for j in range(min(k, len(cand) - 1)):
            note(t, c[t, cand[j]], c[t, cand[j + 1]])
    pj = np.take_along_axis(p, idx.astype(np.int64), 1)
    tot = pj.sum(1, keepdims=True)
    w = s * pj / np.where(tot > 0, tot, 1.0) if renorm else s * pj
    if renorm:
        w = np.where(tot > 0, w, 0.0)
    return idx, w, gap


def permutation(idx, E):
    """off, perm, pos of the stable counting sort by expert."""
    flat = idx.reshape(-1)
    perm = np.argsort(flat, kind="stable").astype(np.int32)
    off = np.zeros(E + 1, np.int32)
    off[1:] = np.cumsum(np.bincount(flat, minlength=E))
    pos = np.empty_like(perm)
    pos[perm] = np.arange(len(flat), dtype=np.int32)
    return off, perm, pos.reshape(idx.shape)
