"""64-bit reference of the balance loss and the router's gradients (numpy), and the error
bounds their fp32 kernels are held to.  Shares no code with the library."""
import numpy as np

from fp8_ref import U32, score

SIGMOID, SQRT_SOFTPLUS, SOFTMAX = 0, 1, 2


def shares(logits, fn):
    """(p, share, relative error of a share in fp32).  Of p: the exponential 2 ulp (and, of
    a difference, its rounding), log1p 2 ulp, a handful of single roundings; of the sum over E:
    eight values a chunk and four chunks in a row, then five levels."""
    l, p = score(logits, fn)
    tot = p.sum(1, keepdims=True)
    share = np.where(tot > 0, p / np.where(tot > 0, tot, 1.0), 0.0)
    eps = np.full(l.shape, 12.0)
    if fn == SOFTMAX:
        top = l.max(1, keepdims=True)
        with np.errstate(invalid="ignore"):
            eps = eps + np.where(np.isfinite(l) & np.isfinite(top), top - l, 0.0)
        # a term beyond e^-87 is subnormal or gone; nothing of it shows beside the others
    return p, share, (eps + eps.max(1, keepdims=True, initial=0, where=share > 1e-30) + 45) * U32


def sequences(T, S, seq, live):
    """Each token's sequence, -1 where it does not count."""
    of = np.full(T, -1)
    bounds = [0, T] if seq is None else seq
    for i in range(S):
        of[bounds[i]:bounds[i + 1]] = i
    if live is not None:
        of[np.asarray(live) == 0] = -1
    return of


def balance(logits, idx, k, fn, S=1, seq=None, live=None, coef=1.0):
    """(counts, tokens, prob, loss, relative bounds of prob and loss)."""
    T, E = logits.shape
    _, share, eps = shares(logits, fn)
    of = sequences(T, S, seq, live)
    counts, tokens, prob = np.zeros((S, E), np.int64), np.zeros(S, np.int64), np.zeros((S, E))
    for t in range(T):
        if of[t] >= 0:
            tokens[of[t]] += 1
            prob[of[t]] += share[t]
            for e in idx[t]:
                if 0 <= e < E:
                    counts[of[t], e] += 1
    n = np.maximum(tokens, 1)[:, None]
    prob = prob / n
    loss = coef / S * (E * counts / (k * n) * prob).sum()
    # sums of positive terms: a CTA's tokens in a row (an eighth of them a warp), the warps, the
    # CTAs; then the loss's own sums over E and S
    e_max = eps[share > 1e-30].max() if (share > 1e-30).any() else 0.0
    rel = e_max + (40 + T / 64 + T / 304 / 8) * U32
    return counts, tokens, prob, loss, rel, rel + (40 + S) * U32


def slopes(logits, fn):
    l, _ = score(logits, fn)
    if fn == SOFTMAX:
        return np.ones_like(l)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if fn == SIGMOID:
            return 1.0 / (1.0 + np.exp(l))
        soft = np.maximum(l, 0) + np.log1p(np.exp(-np.abs(l)))
        return np.where(soft > 0, 0.5 / ((1.0 + np.exp(-l)) * np.where(soft > 0, soft, 1)), 0.5)


def route_backward(logits, idx, k, fn, renorm, s, dw=None, counts=None, tokens=None, dloss=1.0,
                   S=1, seq=None, live=None, coef=1.0):
    """(dlogits, its bound)."""
    T, E = logits.shape
    p, share, eps = shares(logits, fn)
    slope = slopes(logits, fn)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    if counts is not None:
        of = sequences(T, S, seq, live)
        n = np.maximum(tokens, 1)[:, None].astype(np.float64)
        A = dloss * coef / S * E * counts / (k * n * n)
        a = np.where((of >= 0)[:, None], A[of], 0.0)
        dot = (a * share).sum(1, keepdims=True)
        d += share * (a - dot)
        mag += share * (np.abs(a) + (np.abs(a) * share).sum(1, keepdims=True))
    if dw is not None:
        for t in range(T):
            ok = [j for j in range(k) if 0 <= idx[t, j] < E]
            e, g = idx[t, ok], dw[t, ok].astype(np.float64)
            pj = p[t, e]
            if renorm:
                q = pj / pj.sum() if pj.sum() > 0 else 0.0 * pj
                v = s * q * (g - (g * q).sum())
                m = abs(s) * q * (np.abs(g) + (np.abs(g) * q).sum())
            else:
                v, m = s * pj * g, abs(s) * pj * np.abs(g)
                if fn == SOFTMAX:
                    d[t] -= p[t] * v.sum()
                    mag[t] += p[t] * m.sum()
            np.add.at(d[t], e, v)
            np.add.at(mag[t], e, m)
    return d * slope, mag * slope * (3 * eps + (2 * k + 60) * U32)


def combine_backward(dy, o, w, pos):
    """(dw, bound, do, bound); do is NaN in rows that no slot names."""
    T, k = pos.shape
    R, width = o.shape
    dy, o = dy.astype(np.float64), o.astype(np.float64)
    dw, edw = np.zeros((T, k)), np.zeros((T, k))
    do = np.full((R, width), np.nan)
    for t in range(T):
        for j in range(k):
            r = pos[t, j]
            if 0 <= r < R:
                dw[t, j] = o[r] @ dy[t]
                edw[t, j] = np.abs(o[r]) @ np.abs(dy[t]) * (width / 32 + 16) * U32
                do[r] = float(w[t, j]) * dy[t]
    return dw, edw, do, np.abs(do) * U32
