"""Measured cases of the block-scaled fp8 experts and their router.

Five operators, each in a plain form (elementary torch operations in 32 bits)
and, with ``own`` set, through the package's entry points:

  route     group-limited top-k routing of T tokens and the stable permutation
            of their (token, slot) rows by expert
  quantise  rows to e4m3 with one fp32 scale per 128 columns
  swiglu    gate and up products of the routed rows over e4m3 weights with one
            scale per 128 x 128 block, silu(g) * u, quantised like `quantise`
  product   out = rows x weights^T over the same weights (one expert: dense)
  combine   y[t] = shared[t] + sum_j w[t, j] * o[pos[t, j]]
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -100  # smallest block maximum a scale is made from
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


def _blocks(n):
    return -(-n // BLOCK)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a decode step through the router: launch latency alone
        {"name": "route_1", "op": "route", "tokens": 1, "experts": 256, "top_k": 8, "groups": 8,
         "groups_kept": 4, "score": "sigmoid", "bias": True, "type": "float32"},
        # a prefill chunk through the router, logits as a bf16 product leaves them
        {"name": "route_8192", "op": "route", "tokens": 8192, "experts": 256, "top_k": 8,
         "groups": 8, "groups_kept": 4, "score": "sigmoid", "bias": True, "type": "bfloat16"},
        # the hidden state of one token
        {"name": "quantise_1", "op": "quantise", "tokens": 1, "width": 6144, "type": "bfloat16"},
        # the hidden states of a prefill chunk
        {"name": "quantise_8192", "op": "quantise", "tokens": 8192, "width": 6144,
         "type": "bfloat16"},
        # one token, 8 of 256 experts: the weight stream of a decode step
        {"name": "swiglu_1", "op": "swiglu", "tokens": 1, "experts": 256, "top_k": 8,
         "width": 6144, "inner": 2048, "skew": 0.4},
        # 512 tokens over 256 experts: every expert's weights read for about 16 rows
        {"name": "swiglu_512", "op": "swiglu", "tokens": 512, "experts": 256, "top_k": 8,
         "width": 6144, "inner": 2048, "skew": 0.4},
        # a prefill chunk over few experts: about a thousand rows each, bound by arithmetic
        {"name": "swiglu_4096", "op": "swiglu", "tokens": 4096, "experts": 16, "top_k": 4,
         "width": 6144, "inner": 2048, "skew": 0.4},
        # the down projection of a decode step
        {"name": "product_1", "op": "product", "tokens": 1, "experts": 256, "top_k": 8,
         "width": 2048, "out": 6144, "skew": 0.4, "type": "bfloat16"},
        # a small ragged batch, sizes that end inside a block and a tile
        {"name": "product_77", "op": "product", "tokens": 77, "experts": 24, "top_k": 6,
         "width": 1040, "out": 2000, "skew": 0.4, "type": "float32"},
        # a dense projection of a prefill chunk (the shared expert's shape)
        {"name": "product_dense", "op": "product", "tokens": 4000, "experts": 1, "top_k": 1,
         "width": 6144, "out": 4096, "skew": 0.0, "type": "bfloat16"},
        # joining one token's experts
        {"name": "combine_1", "op": "combine", "tokens": 1, "top_k": 8, "width": 6144,
         "shared": True, "type": "bfloat16"},
        # joining a prefill chunk's experts
        {"name": "combine_4096", "op": "combine", "tokens": 4096, "top_k": 8, "width": 6144,
         "shared": True, "type": "bfloat16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A multiple of 16, half of them whole blocks."""
    step = rng.choice((16, BLOCK))
    n = max(step, _log_int(rng, lo, hi) // step * step)
    return n + step if n == 3072 else n


def _tokens(rng, hi, top_k=1):
    t = _log_int(rng, 1, hi)
    return t + 1 if 3072 in (t, t * top_k) else t


def draw(rng):
    op = rng.choice(("route", "quantise", "swiglu", "swiglu", "product", "product", "combine"))
    if op == "route":
        groups = rng.choice((1, 1, 4, 8))
        experts = groups * rng.choice((4, 8, 16, 20, 32, 48))
        top_k = rng.randint(1, min(8, experts // groups))
        score = rng.choice(("sigmoid", "sigmoid", "softmax"))
        # the bias that balances the experts belongs to the sigmoid router
        return {"op": op, "tokens": _tokens(rng, 16384, top_k), "experts": experts,
                "top_k": top_k, "groups": groups, "groups_kept": rng.randint(1, groups),
                "score": score, "bias": score == "sigmoid" and rng.random() < 0.7,
                "type": rng.choice(tuple(DTYPES))}
    if op == "quantise":
        return {"op": op, "tokens": _tokens(rng, 8192), "width": _width(rng, 128, 8192),
                "type": rng.choice(tuple(DTYPES))}
    if op == "combine":
        top_k = rng.randint(1, 8)
        return {"op": op, "tokens": _tokens(rng, 4096, top_k), "top_k": top_k,
                "width": _width(rng, 128, 6144), "shared": rng.random() < 0.5,
                "type": rng.choice(tuple(DTYPES))}
    experts = rng.choice((1, 4, 16, 24, 64, 128, 256))
    top_k = rng.randint(1, min(8, experts))
    # as many tokens as keep a drawn case under the largest listed one
    tokens = _tokens(rng, 16384 // max(4, top_k), top_k)
    case = {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k}
    if op == "swiglu":
        case.update(width=_width(rng, 256, 6144), inner=_width(rng, 128, 2048))
    else:
        case.update(width=_width(rng, 256, 6144), out=_width(rng, 128, 4096),
                    type=rng.choice(tuple(DTYPES)))
    case["skew"] = 0.0 if experts == 1 else rng.choice((0.0, 0.4))
    return case


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)


def _logits(g, tokens, experts, skew):
    """N(0, 1) with a popularity offset that falls with a shuffled rank."""
    rank = torch.randperm(experts, generator=g, device="cuda") + 1
    l = torch.randn((tokens, experts), generator=g, device="cuda")
    return l - skew * 1.1 * torch.log(rank.float())


def _codes(g, rows, cols):
    """e4m3 codes of N(0, 1) values scaled to use the type's range."""
    v = torch.randn((rows, cols), generator=g, device="cuda") * 100.0
    return v.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _weights(g, experts, n, k):
    q = torch.empty((experts, n, k), dtype=torch.float8_e4m3fn, device="cuda")
    for e in range(experts):
        q[e] = _codes(g, n, k)
    s = torch.rand((experts, _blocks(n), _blocks(k)), generator=g, device="cuda")
    return q, (0.5 + s) / (100.0 * math.sqrt(k))


def _rows(g, rows, cols):
    s = torch.rand((rows, _blocks(cols)), generator=g, device="cuda")
    return _codes(g, rows, cols), (0.5 + s) / 100.0


def _assignment(g, case):
    """The experts of T tokens and the stable order of their rows."""
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    idx = _logits(g, T, E, case["skew"]).topk(k, dim=1).indices.reshape(-1)
    perm = torch.argsort(idx, stable=True)
    counts = torch.bincount(idx, minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = counts.cumsum(0)
    return idx[perm], perm.to(torch.int32), off, int(counts.max())


def _inputs(case, seed):
    g = _generator(seed)
    op, T = case["op"], case["tokens"]
    s = {"case": case}
    if op == "route":
        s["logits"] = _logits(g, T, case["experts"], 0.4).to(DTYPES[case["type"]])
        s["bias"] = (0.1 * torch.randn(case["experts"], generator=g, device="cuda")
                     if case["bias"] else None)
    elif op == "quantise":
        x = torch.randn((T, case["width"]), generator=g, device="cuda")
        # a few columns carry values far above the others, as hidden states do
        hot = torch.rand(case["width"], generator=g, device="cuda") < 0.01
        s["x"] = (x * (1.0 + 30.0 * hot)).to(DTYPES[case["type"]])
    elif op == "combine":
        R, k = T * case["top_k"], case["top_k"]
        dt = DTYPES[case["type"]]
        s["o"] = torch.randn((R, case["width"]), generator=g, device="cuda").to(dt)
        w = torch.rand((T, k), generator=g, device="cuda") + 0.05
        s["w"] = 2.5 * w / w.sum(1, keepdim=True)
        s["pos"] = torch.randperm(R, generator=g, device="cuda").to(torch.int32).view(T, k)
        s["shared"] = (torch.randn((T, case["width"]), generator=g, device="cuda").to(dt)
                       if case["shared"] else None)
    else:
        s["expert_of_row"], s["perm"], s["off"], s["most_rows"] = _assignment(g, case)
        E, K = case["experts"], case["width"]
        if op == "swiglu":
            s["xq"], s["xs"] = _rows(g, T, K)
            s["gate"] = _weights(g, E, case["inner"], K)
            s["up"] = _weights(g, E, case["inner"], K)
        else:
            s["xq"], s["xs"] = _rows(g, T * case["top_k"], K)
            s["weight"] = _weights(g, E, case["out"], K)
    return s


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    s = _inputs(case, seed)
    op, T = case["op"], case["tokens"]
    # the buffers that a caller of the package keeps
    if op == "route":
        E, k = case["experts"], case["top_k"]
        s["outputs"] = (_empty((T, k), torch.int32), _empty((T, k), torch.float32),
                        _empty((E + 1,), torch.int32), _empty((T * k,), torch.int32),
                        _empty((T, k), torch.int32))
    elif op == "quantise":
        s["outputs"] = (_empty((T, case["width"]), torch.float8_e4m3fn),
                        _empty((T, _blocks(case["width"])), torch.float32))
    elif op == "combine":
        s["outputs"] = _empty((T, case["width"]), DTYPES[case["type"]])
    elif op == "swiglu":
        R = T * case["top_k"]
        s["outputs"] = (_empty((R, case["inner"]), torch.float8_e4m3fn),
                        _empty((R, _blocks(case["inner"])), torch.float32))
    else:
        s["outputs"] = _empty((T * case["top_k"], case["out"]), DTYPES[case["type"]])
    if own:
        from routed_expert_decode_gb300 import fp8

        need = 0
        if op == "route":
            s["router"] = fp8.make_router(
                case["experts"], case["top_k"], n_group=case["groups"],
                topk_group=case["groups_kept"],
                score=fp8.SCORE_SIGMOID if case["score"] == "sigmoid" else fp8.SCORE_SOFTMAX,
                group_score=fp8.GROUP_TOP2_SUM if case["score"] == "sigmoid" else fp8.GROUP_MAX,
                renorm=True, s=2.5)
            need = fp8.group_route_workspace_size(s["router"], T)
        elif op in ("swiglu", "product"):
            need = fp8.workspace_size(T * case["top_k"])
            for name in ("gate", "up", "weight"):
                if name in s:
                    s[name] = fp8.Mat(*s[name])
        if need:
            s["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    from routed_expert_decode_gb300 import fp8

    case, out = s["case"], s["outputs"]
    op = case["op"]
    if op == "route":
        fp8.group_route(s["router"], s["logits"], s["bias"], *out, s["ws"])
    elif op == "quantise":
        fp8.quantize(s["x"], *out)
    elif op == "swiglu":
        fp8.swiglu(s["gate"], s["up"], s["xq"], s["xs"], *out, s["ws"], off=s["off"],
                   perm=s["perm"], top_k=case["top_k"])
    elif op == "product":
        off = s["off"] if case["experts"] > 1 else None
        fp8.product(s["weight"], s["xq"], s["xs"], out, s["ws"], off=off)
    else:
        fp8.combine(s["o"], s["w"], s["pos"], out, shared=s["shared"])
    return out


def _plain_route(s):
    case = s["case"]
    E, k, G = case["experts"], case["top_k"], case["groups"]
    l = s["logits"].float()
    T = l.shape[0]
    if case["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
        c = p
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        c = l  # softmax keeps the order of the logits
    if s["bias"] is not None:
        c = c + s["bias"]
    by_group = c.view(T, G, E // G)
    if case["score"] == "sigmoid":  # a group's score: its two best experts, or its best
        score = by_group.sort(dim=2, descending=True).values[:, :, :2].sum(2)
    else:
        score = by_group.amax(2)
    kept = score.sort(dim=1, descending=True, stable=True).indices[:, :case["groups_kept"]]
    mask = torch.zeros((T, G), dtype=torch.bool, device="cuda").scatter_(1, kept, True)
    c = c.masked_fill(~mask.repeat_interleave(E // G, 1), float("-inf"))
    idx = c.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, idx)
    w = 2.5 * w / w.sum(1, keepdim=True)
    flat = idx.reshape(-1)
    perm = torch.argsort(flat, stable=True)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.zeros(E, dtype=torch.int32, device="cuda").scatter_add_(
        0, flat, torch.ones_like(flat, dtype=torch.int32)).cumsum(0)
    pos = torch.empty_like(perm).scatter_(0, perm, torch.arange(T * k, device="cuda"))
    return (idx.to(torch.int32), w, off, perm.to(torch.int32), pos.to(torch.int32).view(T, k))


def _plain_quantised(x):
    """e4m3 codes and scales of float32 rows, one scale per 128 columns."""
    T, n = x.shape
    padded = torch.zeros((T, _blocks(n) * BLOCK), device="cuda")
    padded[:, :n] = x
    b = padded.view(T, -1, BLOCK)
    a = b.abs().amax(2).clamp_min(AMAX_MIN)
    q = (b * (E4M3_MAX / a)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.view(T, -1)[:, :n].to(torch.float8_e4m3fn), a / E4M3_MAX


def _plain_quantise(s):
    return _plain_quantised(s["x"].float())


def _spread(scale, n):
    """Scales of blocks of 128 along the last dimension, for n values."""
    return scale.repeat_interleave(BLOCK, -1)[..., :n]


def _plain_rows_by_weights(x, weight, s):
    """Rows in expert order times their expert's weights, transposed."""
    q, scale = weight
    E, N, K = q.shape
    rows = x.shape[0]
    if rows <= E:  # few rows: their experts' weights, row by row
        q = q.view(torch.uint8)[s["expert_of_row"]].view(torch.float8_e4m3fn)
        scale = scale[s["expert_of_row"]]
    w = q.float() * _spread(_spread(scale, K).transpose(1, 2), N).transpose(1, 2)
    if rows <= E:
        return torch.bmm(w, x[:, :, None])[:, :, 0]
    # every expert's rows in a slab of its own, as many as the fullest expert has
    at = torch.arange(rows, device="cuda") - s["off"][s["expert_of_row"]]
    slab = torch.zeros((E, s["most_rows"], K), device="cuda")
    slab[s["expert_of_row"], at] = x
    return torch.bmm(slab, w.transpose(1, 2))[s["expert_of_row"], at]


def _plain_swiglu(s):
    x = s["xq"].float() * _spread(s["xs"], s["xq"].shape[1])
    x = x[s["perm"] // s["case"]["top_k"]]
    g = _plain_rows_by_weights(x, s["gate"], s)
    u = _plain_rows_by_weights(x, s["up"], s)
    return _plain_quantised(g / (1.0 + torch.exp(-g)) * u)


def _plain_product(s):
    x = s["xq"].float() * _spread(s["xs"], s["xq"].shape[1])
    return _plain_rows_by_weights(x, s["weight"], s).to(DTYPES[s["case"]["type"]])


def _plain_combine(s):
    y = (s["o"][s["pos"]].float() * s["w"][:, :, None]).sum(1)
    if s["shared"] is not None:
        y = s["shared"].float() + y
    return y.to(s["o"].dtype)


_PLAIN = {"route": _plain_route, "quantise": _plain_quantise, "swiglu": _plain_swiglu,
          "product": _plain_product, "combine": _plain_combine}


# ------------------------------------------------------------------ work
def work(case):
    """Bytes read and written once, and the arithmetic that the formulas ask for."""
    op, T = case["op"], case["tokens"]
    size = {"float32": 4, "bfloat16": 2, "float16": 2}.get(case.get("type"), 0)
    if op == "route":
        E, k = case["experts"], case["top_k"]
        return {"bytes": T * E * size + 4 * E + 4 * (E + 1) + 16 * T * k, "flops": 10.0 * T * E}
    if op == "quantise":
        d = case["width"]
        return {"bytes": T * (d * (size + 1) + 4 * _blocks(d)), "flops": 3.0 * T * d}
    if op == "combine":
        d, k = case["width"], case["top_k"]
        return {"bytes": T * (d * size * (k + 1 + case["shared"]) + 8 * k),
                "flops": 2.0 * T * k * d}
    # the experts that any row goes to: E (1 - (1 - k/E)^T) of them at even odds
    E, k, K = case["experts"], case["top_k"], case["width"]
    live = E * (1.0 - (1.0 - k / E) ** T)
    R = T * k
    if op == "swiglu":
        N = case["inner"]
        weights = 2 * live * (N * K + 4 * _blocks(N) * _blocks(K))
        return {"bytes": weights + T * (K + 4 * _blocks(K)) + R * (N + 4 * _blocks(N) + 4),
                "flops": 4.0 * R * N * K}
    N = case["out"]
    weights = live * (N * K + 4 * _blocks(N) * _blocks(K))
    return {"bytes": weights + R * (K + 4 * _blocks(K) + N * size), "flops": 2.0 * R * N * K}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    with torch.no_grad():
        return _EXACT[case["op"]](case, s)


def _exact_route(case, s):
    l = s["logits"].double()
    k, E, G = case["top_k"], case["experts"], case["groups"]
    p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    c = p if s["bias"] is None else p + s["bias"].double()
    best = c.unflatten(1, (G, E // G)).topk(min(2 if case["score"] == "sigmoid" else 1, E // G), 2)
    groups = best.values.sum(2).topk(case["groups_kept"], 1).indices
    of_expert = torch.arange(E, device="cuda") // (E // G)
    allowed = (of_expert[None, :, None] == groups[:, None, :]).any(2)
    idx = torch.where(allowed, c, -math.inf).topk(k, 1).indices
    w = torch.take_along_dim(p, idx, 1)
    return (None, 2.5 * w / w.sum(1, keepdim=True), None, None, None)


def _exact_e4m3(v):
    """v rounded to the nearest e4m3 value, ties to even, in 64 bits."""
    exponent = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -30))).clamp(min=-6.0)
    step = torch.exp2(exponent - 3.0)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_quantised(x):
    pad = (-x.shape[1]) % BLOCK
    b = torch.nn.functional.pad(x, (0, pad)).unflatten(1, (-1, BLOCK))
    a = torch.maximum(b.abs().max(dim=2).values, torch.tensor(AMAX_MIN).double().cuda())
    q = _exact_e4m3(b / a[..., None] * E4M3_MAX).flatten(1)
    return q[:, :x.shape[1]], a / E4M3_MAX


def _exact_quantise(case, s):
    return _exact_quantised(s["x"].double())


def _exact_matrix(q, scale):
    """A 64-bit matrix from its codes and its scales' last two dimensions."""
    n = torch.arange(q.shape[0], device="cuda")
    k = torch.arange(q.shape[1], device="cuda") // BLOCK
    return q.double() * scale.double()[n // BLOCK][:, k]


def _exact_by_expert(case, s, one):
    """one(expert, rows of x in 64 bits) for each expert with rows, in order."""
    x = s["xq"].double() * s["xs"].double()[:, torch.arange(case["width"], device="cuda") // BLOCK]
    bounds = s["off"].tolist()
    parts = []
    for e in range(case["experts"]):
        if bounds[e + 1] > bounds[e]:
            r = torch.arange(bounds[e], bounds[e + 1], device="cuda")
            if case["op"] == "swiglu":
                r = s["perm"][r].long() // case["top_k"]
            parts.append(one(e, x[r]))
    return torch.cat(parts)


def _exact_swiglu(case, s):
    def one(e, x):
        g = x @ _exact_matrix(s["gate"][0][e], s["gate"][1][e]).T
        u = x @ _exact_matrix(s["up"][0][e], s["up"][1][e]).T
        return g * torch.sigmoid(g) * u

    return _exact_quantised(_exact_by_expert(case, s, one))


def _exact_product(case, s):
    q, scale = s["weight"]
    return _exact_by_expert(case, s, lambda e, x: x @ _exact_matrix(q[e], scale[e]).T)


def _exact_combine(case, s):
    y = torch.zeros((case["tokens"], case["width"]), dtype=torch.float64, device="cuda")
    for j in range(case["top_k"]):
        y += s["w"][:, j, None].double() * s["o"][s["pos"][:, j].long()].double()
    return y if s["shared"] is None else y + s["shared"].double()


_EXACT = {"route": _exact_route, "quantise": _exact_quantise, "swiglu": _exact_swiglu,
          "product": _exact_product, "combine": _exact_combine}
