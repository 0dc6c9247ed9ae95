"""Measured cases of the int8 experts and of the gradients that train a router over them.

Five operators, each in a plain form (elementary torch operations in 32 bits)
and, with ``own`` set, through the package's entry points:

  product       out = rows x weights^T over int8 codes with one scale per row and one
                per weight channel, routed by expert or dense; with ``raw`` the rows
                come in a floating type and are quantised first, as a program does
  swiglu        gate and up products of the routed rows, silu(g) * u
  balance       per-expert counts and mean probabilities of each sequence's tokens,
                and the loss that evens them out
  route_grad    the logits' gradient from the routing weights' and that loss's
  combine_grad  gradients of y[t] = sum_j w[t, j] * o[pos[t, j]]
"""
import math

import torch

own = False

CODE_MAX = 127.0
AMAX_MIN = 2.0 ** -100  # smallest row maximum a scale is made from
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SCORES = ("sigmoid", "sqrt_softplus", "softmax")
ROUTE_SCALE = 2.5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the down projection of a decode step: one token, 8 of 256 experts
        {"name": "product_1", "op": "product", "tokens": 1, "experts": 256, "top_k": 8,
         "width": 2048, "out": 6144, "skew": 0.4, "raw": False, "type": "bfloat16"},
        # a small ragged batch, sizes that end inside a tile
        {"name": "product_77", "op": "product", "tokens": 77, "experts": 24, "top_k": 6,
         "width": 1040, "out": 2000, "skew": 0.4, "raw": False, "type": "float32"},
        # a dense projection of a prefill chunk, hidden states as they come
        {"name": "product_dense", "op": "product", "tokens": 4000, "experts": 1, "top_k": 1,
         "width": 6144, "out": 4096, "skew": 0.0, "raw": True, "type": "bfloat16"},
        # gate and up of a decode step: the weight stream of one token
        {"name": "swiglu_1", "op": "swiglu", "tokens": 1, "experts": 256, "top_k": 8,
         "width": 6144, "inner": 2048, "skew": 0.4, "type": "bfloat16"},
        # 512 tokens over 256 experts: every expert's weights read for about 16 rows
        {"name": "swiglu_512", "op": "swiglu", "tokens": 512, "experts": 256, "top_k": 8,
         "width": 6144, "inner": 2048, "skew": 0.4, "type": "bfloat16"},
        # a prefill chunk over few experts: about a thousand rows each, bound by arithmetic
        {"name": "swiglu_4096", "op": "swiglu", "tokens": 4096, "experts": 16, "top_k": 4,
         "width": 6144, "inner": 2048, "skew": 0.4, "type": "bfloat16"},
        # a short calibration batch through the balance loss
        {"name": "balance_100", "op": "balance", "tokens": 100, "experts": 64, "top_k": 6,
         "sequences": 1, "padded": False, "score": "softmax", "type": "float32"},
        # a training micro-batch: 16 sequences of different lengths, some tokens padding
        {"name": "balance_65536", "op": "balance", "tokens": 65536, "experts": 256, "top_k": 8,
         "sequences": 16, "padded": True, "score": "sigmoid", "type": "bfloat16"},
        # the same two batches on the way back
        {"name": "route_grad_100", "op": "route_grad", "tokens": 100, "experts": 64, "top_k": 6,
         "sequences": 1, "padded": False, "score": "softmax", "renorm": False,
         "type": "float32"},
        {"name": "route_grad_65536", "op": "route_grad", "tokens": 65536, "experts": 256,
         "top_k": 8, "sequences": 16, "padded": True, "score": "sigmoid", "renorm": True,
         "type": "bfloat16"},
        # what a layer's output gradient says of its experts' outputs and their weights
        {"name": "combine_grad_100", "op": "combine_grad", "tokens": 100, "top_k": 6,
         "width": 2000, "type": "float32"},
        {"name": "combine_grad_4096", "op": "combine_grad", "tokens": 4096, "top_k": 8,
         "width": 6144, "type": "bfloat16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A multiple of 16, half of them of 128."""
    step = rng.choice((16, 128))
    return max(step, _log_int(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(("product", "product", "swiglu", "swiglu", "balance", "route_grad",
                     "combine_grad"))
    kind = rng.choice(tuple(DTYPES))
    if op in ("balance", "route_grad"):
        experts = rng.choice((8, 20, 32, 64, 96, 160, 192, 256, 384))
        tokens = _log_int(rng, 1, 65536 * 256 // max(256, experts))
        case = {"op": op, "tokens": tokens, "experts": experts, "top_k": rng.randint(1, 8),
                "sequences": _log_int(rng, 1, min(64, tokens)), "padded": rng.random() < 0.5,
                "score": rng.choice(SCORES), "type": kind}
        if op == "route_grad":
            case["renorm"] = rng.random() < 0.7
        return case
    if op == "combine_grad":
        # 32-bit values are twice the bytes of the largest listed case's
        return {"op": op, "tokens": _log_int(rng, 1, 2048 if kind == "float32" else 4096),
                "top_k": rng.randint(1, 8), "width": _width(rng, 128, 6144), "type": kind}
    experts = rng.choice((1, 4, 16, 24, 64, 128, 256))
    top_k = rng.randint(1, min(8, experts))
    # as many tokens as keep a drawn case under the largest listed one
    case = {"op": op, "tokens": _log_int(rng, 1, 16384 // max(4, top_k)), "experts": experts,
            "top_k": top_k, "width": _width(rng, 256, 6144),
            "skew": 0.0 if experts == 1 else rng.choice((0.0, 0.4)), "type": kind}
    if op == "swiglu":
        case["inner"] = _width(rng, 128, 2048)
    else:
        case.update(out=_width(rng, 128, 4096), raw=rng.random() < 0.4)
    return case


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 6007 + 29)


def _logits(g, tokens, experts, skew):
    """N(0, 1) with a popularity offset that falls with a shuffled rank."""
    rank = torch.randperm(experts, generator=g, device="cuda") + 1
    l = torch.randn((tokens, experts), generator=g, device="cuda")
    return l - skew * 1.1 * torch.log(rank.float())


def _codes(g, rows, cols):
    """int8 codes of N(0, 1) values, four deviations wide."""
    v = torch.randn((rows, cols), generator=g, device="cuda") * 32.0
    return v.round_().clamp_(-CODE_MAX, CODE_MAX).to(torch.int8)


def _weights(g, experts, n, k):
    q = torch.empty((experts, n, k), dtype=torch.int8, device="cuda")
    for e in range(experts):
        q[e] = _codes(g, n, k)
    s = torch.rand((experts, n), generator=g, device="cuda")
    return q, (0.5 + s) / (32.0 * math.sqrt(k))


def _rows(g, rows, cols):
    s = torch.rand((rows,), generator=g, device="cuda")
    return _codes(g, rows, cols), (0.5 + s) / 32.0


def _hidden(g, rows, cols, kind):
    """Hidden states: a few columns carry values far above the others."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    hot = torch.rand(cols, generator=g, device="cuda") < 0.01
    return (x * (1.0 + 30.0 * hot)).to(DTYPES[kind])


def _assignment(g, case):
    """The experts of T tokens and the stable order of their rows."""
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    idx = _logits(g, T, E, case["skew"]).topk(k, dim=1).indices.reshape(-1)
    perm = torch.argsort(idx, stable=True)
    counts = torch.bincount(idx, minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = counts.cumsum(0)
    return idx[perm], perm.to(torch.int32), off, int(counts.max())


def _batch(g, case):
    """Router logits of a batch of sequences, its picks, and which tokens count."""
    T, E, S = case["tokens"], case["experts"], case["sequences"]
    s = {"logits": _logits(g, T, E, 0.4).to(DTYPES[case["type"]])}
    s["idx"] = s["logits"].float().topk(case["top_k"], dim=1).indices.to(torch.int32)
    # sequences of uneven lengths; a padded batch ends behind the last of them
    end = max(S, T - T // 16) if case["padded"] else T
    cuts = (torch.randperm(end - 1, generator=g, device="cuda")[:S - 1] + 1 if S > 1
            else torch.zeros(0, dtype=torch.int64, device="cuda"))
    seq = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    seq[1:S] = cuts.sort().values
    seq[S] = end
    s["seq"] = seq
    s["live"] = ((torch.rand(T, generator=g, device="cuda") > 0.1).to(torch.uint8)
                 if case["padded"] else None)
    s["coef"] = 0.01
    return s


def _sequence_of(seq, T):
    """Each token's sequence, S for the tokens behind the last one."""
    return torch.searchsorted(seq[1:].contiguous(), torch.arange(T, device="cuda").int(),
                              right=True)


def _counting(s, T):
    """Each token's sequence and whether it counts."""
    S = s["seq"].shape[0] - 1
    of = _sequence_of(s["seq"], T)
    counting = of < S
    if s["live"] is not None:
        counting = counting & (s["live"] != 0)
    return of.clamp(max=S - 1), counting


def _counts(s, T, E):
    S = s["seq"].shape[0] - 1
    of, counting = _counting(s, T)
    n = torch.zeros(S, dtype=torch.int32, device="cuda").scatter_add_(0, of, counting.int())
    at = (of[:, None] * E + s["idx"]).reshape(-1)
    ones = counting.int()[:, None].expand_as(s["idx"]).reshape(-1)
    c = torch.zeros(S * E, dtype=torch.int32, device="cuda").scatter_add_(0, at, ones)
    return c.view(S, E), n


def _inputs(case, seed):
    g = _generator(seed)
    op, T = case["op"], case["tokens"]
    s = {"case": case}
    if op in ("balance", "route_grad"):
        s.update(_batch(g, case))
        if op == "route_grad":
            s["counts"], s["live_tokens"] = _counts(s, T, case["experts"])
            s["dw"] = torch.randn((T, case["top_k"]), generator=g, device="cuda") / T
            s["dloss"] = torch.full((1,), 1.5, device="cuda")
    elif op == "combine_grad":
        R, k, dt = T * case["top_k"], case["top_k"], DTYPES[case["type"]]
        s["o"] = torch.randn((R, case["width"]), generator=g, device="cuda").to(dt)
        s["dy"] = torch.randn((T, case["width"]), generator=g, device="cuda").to(dt)
        w = torch.rand((T, k), generator=g, device="cuda") + 0.05
        s["w"] = ROUTE_SCALE * w / w.sum(1, keepdim=True)
        s["pos"] = torch.randperm(R, generator=g, device="cuda").to(torch.int32).view(T, k)
    else:
        s["expert_of_row"], s["perm"], s["off"], s["most_rows"] = _assignment(g, case)
        E, K, k = case["experts"], case["width"], case["top_k"]
        if op == "swiglu":
            s["xq"], s["xs"] = _rows(g, T, K)
            s["gate"] = _weights(g, E, case["inner"], K)
            s["up"] = _weights(g, E, case["inner"], K)
        else:
            if case["raw"]:
                s["x"] = _hidden(g, T * k, K, case["type"])
            else:
                s["xq"], s["xs"] = _rows(g, T * k, K)
            s["weight"] = _weights(g, E, case["out"], K)
    return s


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    s = _inputs(case, seed)
    op, T = case["op"], case["tokens"]
    dt = DTYPES[case["type"]]
    # the buffers that a caller of the package keeps
    if op == "balance":
        S, E = case["sequences"], case["experts"]
        s["outputs"] = (_empty((S, E), torch.int32), _empty((S,), torch.int32),
                        _empty((S, E), torch.float32), _empty((1,), torch.float32))
    elif op == "route_grad":
        s["outputs"] = _empty((T, case["experts"]), dt)
    elif op == "combine_grad":
        R = T * case["top_k"]
        s["outputs"] = (_empty((T, case["top_k"]), torch.float32), _empty((R, case["width"]), dt))
    else:
        R = T * case["top_k"]
        s["outputs"] = _empty((R, case["inner"] if op == "swiglu" else case["out"]), dt)
        if case.get("raw"):
            s["codes"] = (_empty((R, case["width"]), torch.int8), _empty((R,), torch.float32))
    if own:
        from routed_expert_decode_gb300 import fp8, int8, router_grad

        need = 0
        if op in ("balance", "route_grad"):
            score = (fp8.SCORE_SIGMOID, fp8.SCORE_SQRT_SOFTPLUS,
                     fp8.SCORE_SOFTMAX)[SCORES.index(case["score"])]
            s["router"] = fp8.make_router(case["experts"], case["top_k"], score=score,
                                          renorm=case.get("renorm", True), s=ROUTE_SCALE)
            if op == "balance":
                need = router_grad.workspace_size(s["router"], T, case["sequences"])
        elif op in ("swiglu", "product"):
            need = int8.workspace_size(T * case["top_k"])
            for name in ("gate", "up", "weight"):
                if name in s:
                    s[name] = int8.Mat(*s[name])
        if need:
            s["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    from routed_expert_decode_gb300 import int8, router_grad

    case, out = s["case"], s["outputs"]
    op = case["op"]
    if op == "swiglu":
        int8.swiglu(s["gate"], s["up"], s["xq"], s["xs"], out, s["ws"], off=s["off"],
                    perm=s["perm"], top_k=case["top_k"])
    elif op == "product":
        off = s["off"] if case["experts"] > 1 else None
        if case["raw"]:
            xq, xs = s["codes"]
            int8.quantize(s["x"], xq, xs)
        else:
            xq, xs = s["xq"], s["xs"]
        int8.product(s["weight"], xq, xs, out, s["ws"], off=off)
    elif op == "balance":
        router_grad.balance(s["router"], s["logits"], s["idx"], *out, s["ws"], seq=s["seq"],
                            live=s["live"], coef=s["coef"])
    elif op == "route_grad":
        router_grad.route_backward(s["router"], s["logits"], s["idx"], out, dw=s["dw"],
                                   counts=s["counts"], tokens=s["live_tokens"], dloss=s["dloss"],
                                   seq=s["seq"], live=s["live"], coef=s["coef"])
    else:
        router_grad.combine_backward(s["dy"], s["o"], s["w"], s["pos"], *out)
    return out


def _plain_codes(x):
    """int8 codes and scales of rows, one scale a row."""
    x = x.float()
    a = x.abs().amax(1, keepdim=True).clamp_min(AMAX_MIN)
    # quotients of two tensors: one by a number would be a product with its reciprocal
    top = torch.full_like(a, CODE_MAX)
    return (x * (top / a)).round(), (a / top)[:, 0]


def _plain_rows_by_weights(x, weight, s):
    """Rows in expert order times their expert's weights, transposed: sums of codes."""
    q, scale = weight
    E, N, K = q.shape
    rows = x.shape[0]
    if rows <= E:  # few rows: their experts' weights, row by row
        w = q[s["expert_of_row"]].float()
        return torch.bmm(w, x[:, :, None])[:, :, 0] * scale[s["expert_of_row"]]
    # every expert's rows in a slab of its own, as many as the fullest expert has
    at = torch.arange(rows, device="cuda") - s["off"][s["expert_of_row"]]
    slab = torch.zeros((E, s["most_rows"], K), device="cuda")
    slab[s["expert_of_row"], at] = x
    y = torch.bmm(slab, q.float().transpose(1, 2)) * scale[:, None, :]
    return y[s["expert_of_row"], at]


def _plain_swiglu(s):
    of = s["perm"] // s["case"]["top_k"]
    x, scale = s["xq"].float()[of], s["xs"][of, None]
    g = _plain_rows_by_weights(x, s["gate"], s) * scale
    u = _plain_rows_by_weights(x, s["up"], s) * scale
    return (g / (1.0 + torch.exp(-g)) * u).to(DTYPES[s["case"]["type"]])


def _plain_product(s):
    x, scale = (_plain_codes(s["x"]) if s["case"]["raw"] else (s["xq"].float(), s["xs"]))
    y = _plain_rows_by_weights(x, s["weight"], s) * scale[:, None]
    return y.to(DTYPES[s["case"]["type"]])


def _plain_scores(l, score):
    """(p, slope): the experts' scores and d(log p)/dl, softmax's without its sum's part."""
    if score == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True), torch.ones_like(l)
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l)), 1.0 / (1.0 + torch.exp(l))
    soft = l.clamp(min=0.0) + torch.log1p(torch.exp(-l.abs()))
    return torch.sqrt(soft), 0.5 / ((1.0 + torch.exp(-l)) * soft)


def _plain_balance(s):
    case = s["case"]
    T, E, k, S = case["tokens"], case["experts"], case["top_k"], case["sequences"]
    p, _ = _plain_scores(s["logits"].float(), case["score"])
    if case["score"] != "softmax":
        p = p / p.sum(1, keepdim=True)
    of, counting = _counting(s, T)
    counts, n = _counts(s, T, E)
    # sums over up to all tokens: in 64 bits
    p = torch.where(counting[:, None], p, 0.0).double()
    share = torch.zeros((S, E), dtype=torch.float64, device="cuda").index_add_(0, of, p)
    some = n.clamp(min=1)[:, None].double()
    prob = share / some
    load = counts * (E / k) / some
    loss = s["coef"] / S * (load * prob).sum()
    return counts, n, prob.float(), loss.float().view(1)


def _plain_route_grad(s):
    case = s["case"]
    T, E, k, S = case["tokens"], case["experts"], case["top_k"], case["sequences"]
    p, slope = _plain_scores(s["logits"].float(), case["score"])
    softmax = case["score"] == "softmax"
    share = p if softmax else p / p.sum(1, keepdim=True)
    # the balance loss: d loss / d share, the same for all tokens of a sequence
    n = s["live_tokens"].clamp(min=1)[:, None].float()
    by_sequence = s["dloss"] * (s["coef"] / S * E / k) * s["counts"] / (n * n)
    of, counting = _counting(s, T)
    a = torch.where(counting[:, None], by_sequence[of], 0.0)
    d = share * (a - (a * share).sum(1, keepdim=True))
    # the routing weights, w_j = c p_j / sum p or c p_j
    idx = s["idx"].long()
    pj, dw = p.gather(1, idx), s["dw"]
    if case["renorm"]:
        part = pj / pj.sum(1, keepdim=True)
        v = ROUTE_SCALE * part * (dw - (dw * part).sum(1, keepdim=True))
    else:
        v = ROUTE_SCALE * pj * dw
        if softmax:
            d = d - p * v.sum(1, keepdim=True)
    d = d.scatter_add(1, idx, v)
    return (d * slope).to(DTYPES[case["type"]])


def _plain_combine_grad(s):
    T, k = s["pos"].shape
    dy = s["dy"].float()
    dw = (s["o"][s["pos"]].float() * dy[:, None, :]).sum(2)
    do = torch.empty_like(s["o"])
    do[s["pos"].view(-1)] = (s["w"][:, :, None] * dy[:, None, :]).view(T * k, -1).to(do.dtype)
    return dw, do


_PLAIN = {"product": _plain_product, "swiglu": _plain_swiglu, "balance": _plain_balance,
          "route_grad": _plain_route_grad, "combine_grad": _plain_combine_grad}


# ------------------------------------------------------------------ work
def work(case):
    """Bytes read and written once, and the arithmetic that the formulas ask for."""
    op, T, k = case["op"], case["tokens"], case["top_k"]
    size = 4 if case["type"] == "float32" else 2
    if op in ("balance", "route_grad"):
        E, S = case["experts"], case["sequences"]
        once = T * E * size + 4 * T * k + 4 * (S + 1) + case["padded"] * T
        if op == "balance":
            return {"bytes": once + 8 * S * E + 4 * S + 4, "flops": 8.0 * T * E}
        return {"bytes": once + T * E * size + 4 * T * k + 4 * S * E + 4 * S,
                "flops": 14.0 * T * E}
    if op == "combine_grad":
        d = case["width"]
        return {"bytes": T * (d * size * (2 * k + 1) + 12 * k), "flops": 3.0 * T * k * d}
    # the experts that any row goes to: E (1 - (1 - k/E)^T) of them at even odds
    E, K = case["experts"], case["width"]
    live = E * (1.0 - (1.0 - k / E) ** T)
    R = T * k
    if op == "swiglu":
        N = case["inner"]
        return {"bytes": 2 * live * N * (K + 4) + T * (K + 4) + R * (N * size + 4),
                "flops": 4.0 * R * N * K}
    N = case["out"]
    row = K * size if case["raw"] else K + 4
    return {"bytes": live * N * (K + 4) + R * (row + N * size), "flops": 2.0 * R * N * K}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    return _EXACT[case["op"]](case, s)


def _exact_by_expert(case, s, one):
    """one(expert, codes of its rows in 64 bits, their scales), experts in order."""
    if case.get("raw"):
        x = s["x"].double()
        scale = x.abs().max(dim=1).values.clamp(min=AMAX_MIN) / CODE_MAX
        codes = torch.round(x / scale[:, None])
    else:
        codes, scale = s["xq"].double(), s["xs"].double()
    bounds = s["off"].tolist()
    parts = []
    for e in range(case["experts"]):
        if bounds[e + 1] > bounds[e]:
            r = torch.arange(bounds[e], bounds[e + 1], device="cuda")
            if case["op"] == "swiglu":
                r = s["perm"][r].long() // case["top_k"]
            parts.append(one(e, codes[r] * scale[r, None]))
    return torch.cat(parts)


def _exact_matrix(weight, e):
    q, scale = weight
    return q[e].double() * scale[e].double()[:, None]


def _exact_product(case, s):
    return _exact_by_expert(case, s, lambda e, x: x @ _exact_matrix(s["weight"], e).T)


def _exact_swiglu(case, s):
    def one(e, x):
        g = x @ _exact_matrix(s["gate"], e).T
        return g * torch.sigmoid(g) * (x @ _exact_matrix(s["up"], e).T)

    return _exact_by_expert(case, s, one)


def _exact_scores(case, l):
    if case["score"] == "softmax":
        return torch.softmax(l, 1)
    return (torch.sigmoid(l) if case["score"] == "sigmoid"
            else torch.nn.functional.softplus(l, threshold=700.0).sqrt())


def _exact_loss(case, s, p):
    """(mean probabilities [S, E], loss), sequence by sequence."""
    E, k, S = case["experts"], case["top_k"], case["sequences"]
    share = p / p.sum(1, keepdim=True)
    bounds = s["seq"].tolist()
    probs, loss = [], 0.0
    for a, b in zip(bounds, bounds[1:]):
        rows = torch.arange(a, b, device="cuda")
        if s["live"] is not None:
            rows = rows[s["live"][rows] != 0]
        n = max(1, rows.numel())
        picked = torch.bincount(s["idx"][rows].reshape(-1).long(), minlength=E).double()
        probs.append(share[rows].sum(0) / n)
        loss = loss + (picked * E / (k * n) * probs[-1]).sum()
    return torch.stack(probs), s["coef"] / S * loss


def _exact_balance(case, s):
    prob, loss = _exact_loss(case, s, _exact_scores(case, s["logits"].double()))
    return None, None, prob, loss.view(1)


def _exact_route_grad(case, s):
    with torch.enable_grad():
        l = s["logits"].double().requires_grad_()
        p = _exact_scores(case, l)
        w = torch.take_along_dim(p, s["idx"].long(), 1) * ROUTE_SCALE
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True) * ROUTE_SCALE
        total = (w * s["dw"].double()).sum() + s["dloss"].double() * _exact_loss(case, s, p)[1]
        return torch.autograd.grad(total.sum(), l)[0]


def _exact_combine_grad(case, s):
    T, k = s["pos"].shape
    dy = s["dy"].double()
    dw = torch.empty((T, k), dtype=torch.float64, device="cuda")
    do = torch.empty(s["o"].shape, dtype=torch.float64, device="cuda")
    for j in range(k):
        r = s["pos"][:, j].long()
        dw[:, j] = torch.einsum("td,td->t", s["o"][r].double(), dy)
        do[r] = s["w"][:, j, None].double() * dy
    return dw, do


_EXACT = {"product": _exact_product, "swiglu": _exact_swiglu, "balance": _exact_balance,
          "route_grad": _exact_route_grad, "combine_grad": _exact_combine_grad}
