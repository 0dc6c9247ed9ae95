"""The balance loss and the router's gradients on a GPU against the 64-bit reference, within
the bounds that router_grad_ref derives."""
import numpy as np
import pytest
import torch

import router_grad_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}


@pytest.fixture(scope="module")
def rg(gpu):
    from routed_expert_decode_gb300 import router_grad as m

    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def router(E, k, fn, renorm=True, s=2.5):
    from routed_expert_decode_gb300 import fp8

    return fp8.make_router(E, k, score=fn, renorm=renorm, s=s)


def strided(t, pad):
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


class Batch:
    def __init__(self, T, E, k, S=1, padded=False, dt="f32", seed=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.T, self.E, self.k, self.S = T, E, k, S
        self.logits = dev((rng.standard_normal((T, E)) * spread).astype(np.float32)).to(TYPES[dt])
        self.idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
        self.seq = self.live = None
        if S > 1 or padded:
            cuts = np.sort(rng.integers(0, T + 1, S + 1))  # empty sequences among them
            if not padded:
                cuts[0], cuts[-1] = 0, T
            self.seq = cuts.astype(np.int32)
        if padded:
            self.live = (rng.random(T) > 0.3).astype(np.uint8)
        self.dw = (rng.standard_normal((T, k)) * 0.1).astype(np.float32)

    def where(self):
        return dict(seq=None if self.seq is None else dev(self.seq),
                    live=None if self.live is None else dev(self.live))

    def known(self):
        return dict(S=self.S, seq=self.seq, live=self.live)

    def l(self):
        return self.logits.float().cpu().numpy()


def run_balance(rg, b, fn, coef=1.0, ws=None, logits=None):
    r = router(b.E, b.k, fn)
    out = (torch.full((b.S, b.E), -3, dtype=torch.int32, device="cuda"),
           torch.full((b.S,), -3, dtype=torch.int32, device="cuda"),
           torch.full((b.S, b.E), float("nan"), device="cuda"),
           torch.full((1,), float("nan"), device="cuda"))
    if ws is None:
        ws = torch.zeros(rg.workspace_size(r, b.T, b.S), dtype=torch.uint8, device="cuda")
    rg.balance(r, b.logits if logits is None else logits, dev(b.idx), *out, ws, coef=coef,
               **b.where())
    return out


def check_balance(rg, b, fn, coef=1.0, **kw):
    got = [o.cpu().numpy() for o in run_balance(rg, b, fn, coef, **kw)]
    counts, tokens, prob, loss, e_prob, e_loss = ref.balance(b.l(), b.idx, b.k, fn, coef=coef,
                                                             **b.known())
    assert np.array_equal(got[0], counts) and np.array_equal(got[1], tokens)
    assert (np.abs(got[2] - prob) <= prob * e_prob + 2.0 ** -126).all()
    assert abs(got[3][0] - loss) <= abs(loss) * e_loss + 2.0 ** -126
    return got


SIZES = [(1, 1, 1), (1, 8, 2), (7, 8, 8), (33, 20, 3), (64, 64, 6), (65, 96, 4), (130, 160, 6),
         (300, 256, 8), (100, 257, 5), (90, 384, 6), (77, 512, 8), (50, 1024, 32), (40, 1000, 7),
         (1500, 64, 2)]


@pytest.mark.parametrize("fn", [0, 1, 2])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_balance(rg, T, E, k, fn):
    for dt in TYPES:
        check_balance(rg, Batch(T, E, k, dt=dt, seed=T + E), fn, coef=0.01)


@pytest.mark.parametrize("fn", [0, 2])
@pytest.mark.parametrize("T,E,S", [(40, 64, 7), (700, 32, 3), (700, 256, 40), (3000, 16, 1),
                                   (1000, 8, 1000), (200, 300, 500)])
def test_balance_of_sequences(rg, T, E, S, fn):
    for padded in (False, True):
        check_balance(rg, Batch(T, E, 3, S, padded, seed=S), fn)


@pytest.mark.parametrize("T,S", [(1, 5), (50, 5000), (700, 65535)])
def test_many_empty_sequences(rg, T, S):
    """Runs of empty sequences are passed over (a step each would take tens of ms here)."""
    b = Batch(T, 16, 2, S, seed=S)
    check_balance(rg, b, 0)
    check_backward(rg, b, 0, True)
    b.seq = np.sort(np.concatenate([np.full(S // 2, T // 3), np.full(S - S // 2, T // 2), [T]]))
    b.seq = b.seq.astype(np.int32)  # all of them between two tokens
    check_balance(rg, b, 2)
    check_backward(rg, b, 2, False)


def test_balance_without_tokens(rg):
    b = Batch(20, 16, 2, 4, True)
    b.live[:] = 0
    got = check_balance(rg, b, 0)
    assert not got[0].any() and not got[2].any() and got[3][0] == 0
    b = Batch(0, 16, 2)
    got = check_balance(rg, b, 2)
    assert got[3][0] == 0 and got[1][0] == 0


def special(b):
    l = b.l()
    l[0, :] = -np.inf
    l[1, 3] = np.inf
    l[2, 5] = np.nan
    l[3, :] = np.nan
    l[4, ::2] = -np.inf
    l[5, :] = 3.0e38
    l[6, :] = -3.0e38
    l[7, 1] = -200.0
    b.logits = dev(l)
    return b


@pytest.mark.parametrize("fn", [0, 1, 2])
def test_special_logits(rg, fn):
    b = special(Batch(40, 24, 4, seed=3))
    check_balance(rg, b, fn)
    for renorm in (True, False):
        check_backward(rg, b, fn, renorm)


@pytest.mark.parametrize("fn", [0, 1])
@pytest.mark.parametrize("E", [24, 256])
def test_wide_logits(rg, fn, E):
    """Rows from one end of the scores' range to the other, and rows of its ends alone."""
    b = Batch(48, E, 6, 2, True, seed=14)
    g = np.random.default_rng(15)
    least = -170.0 if fn else -80.0   # whose score is not below the smallest normal float
    l = g.uniform(least, 100.0, (48, E))
    l[:12] = g.uniform(least, least + 40, (12, E))
    l[12:24] = g.uniform(-2.0, 2.0, (12, E))
    l[24:30] = g.uniform(60.0, 100.0, (6, E))
    b.logits = dev(l.astype(np.float32))
    check_balance(rg, b, fn)
    for renorm in (True, False):
        check_backward(rg, b, fn, renorm)


def test_balance_strides_picks_and_repeats(rg):
    b = Batch(500, 64, 4, 6, True, dt="bf16", seed=8)
    b.idx[::7, 1] = -1          # picks that are none
    b.idx[::5, 2] = 64
    b.idx[::3, 3] = b.idx[::3, 0]  # the same expert twice
    want = check_balance(rg, b, 0, logits=strided(b.logits, 8))
    r = router(64, 4, 0)
    ws = torch.zeros(rg.workspace_size(r, 500, 6), dtype=torch.uint8, device="cuda")
    for pad in (0, 3, 8):
        got = check_balance(rg, b, 0, ws=ws, logits=strided(b.logits, pad))
        assert all(np.array_equal(x, y) for x, y in zip(got, want))


# ---------------------------------------------------------------- the logits' gradient
def check_backward(rg, b, fn, renorm, odt="f32", dw=True, loss=True, dloss=1.5, coef=0.02,
                   logits=None, pad=0):
    r = router(b.E, b.k, fn, renorm)
    counts, tokens, *_ = ref.balance(b.l(), b.idx, b.k, fn, **b.known())
    out = torch.full((b.T, b.E + pad), 7.0, dtype=TYPES[odt], device="cuda")
    kw = {}
    if loss:
        kw = dict(counts=dev(counts.astype(np.int32)), tokens=dev(tokens.astype(np.int32)),
                  dloss=None if dloss is None else torch.full((1,), dloss, device="cuda"),
                  coef=coef, **b.where())
    rg.route_backward(r, b.logits if logits is None else logits, dev(b.idx), out[:, :b.E],
                      dw=dev(b.dw) if dw else None, **kw)
    want, bound = ref.route_backward(
        b.l(), b.idx, b.k, fn, renorm, 2.5, b.dw if dw else None, counts if loss else None,
        tokens, 1.0 if dloss is None else dloss, coef=coef, **b.known())
    got = out[:, :b.E].double().cpu().numpy()
    bar = bound + (np.abs(want) + bound) * HALF_ULP[odt] * (odt != "f32") + TINY[odt]
    bad = ~(np.abs(got - want) <= bar)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3],
                           want[bad][:3], bar[bad][:3])
    assert (out[:, b.E:] == 7.0).all()
    return got


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("fn", [0, 1, 2])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_route_backward(rg, T, E, k, fn, renorm):
    for dt in TYPES:
        check_backward(rg, Batch(T, E, k, dt=dt, seed=T + E), fn, renorm, odt=dt)


@pytest.mark.parametrize("parts", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("fn", [0, 1, 2])
def test_route_backward_of_one_part(rg, fn, parts):
    for renorm in (True, False):
        got = check_backward(rg, Batch(70, 40, 5, seed=2), fn, renorm, dw=parts[0], loss=parts[1],
                             dloss=None)
        assert parts != (False, False) or not got.any()


@pytest.mark.parametrize("T,E,S", [(40, 64, 7), (700, 256, 40), (1000, 8, 1000), (3000, 32, 5)])
def test_route_backward_of_sequences(rg, T, E, S):
    for padded in (False, True):
        check_backward(rg, Batch(T, E, 3, S, padded, seed=S), 0, True)


@pytest.mark.parametrize("fn", [0, 2])
@pytest.mark.parametrize("E", [20, 64, 256, 384, 1000])
def test_route_backward_of_many_tokens(rg, E, fn):
    """Warps with many tokens each: every row is what a call of a few hundred tokens gives."""
    T, k, S = 120007 if E < 256 else 30011, 5, 9
    g = torch.Generator("cuda").manual_seed(E)
    logits = torch.randn((T, E), generator=g, device="cuda").to(torch.bfloat16)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    dw = torch.randn((T, k), generator=g, device="cuda")
    live = (torch.rand(T, generator=g, device="cuda") > 0.2).to(torch.uint8)
    seq = dev(np.sort(np.random.default_rng(E).integers(0, T + 1, S + 1)).astype(np.int32))
    counts = torch.randint(0, 900, (S, E), generator=g, device="cuda", dtype=torch.int32)
    tokens = torch.randint(1, 9000, (S,), generator=g, device="cuda", dtype=torch.int32)
    r, got = router(E, k, fn), torch.empty_like(logits)
    rg.route_backward(r, logits, idx, got, dw, counts, tokens, seq=seq, live=live, coef=0.5)
    for a in range(0, T, T // 6):
        n = min(777, T - a)
        few = torch.empty((n, E), dtype=torch.bfloat16, device="cuda")
        rg.route_backward(r, logits[a:a + n], idx[a:a + n], few, dw[a:a + n], counts, tokens,
                          seq=(seq - a).clamp(0, n), live=live[a:a + n], coef=0.5)
        assert torch.equal(got[a:a + n], few), a


def test_route_backward_strides_types_and_picks(rg):
    b = Batch(90, 64, 6, 3, True, seed=8, spread=3.0)
    b.idx[::7, 1] = -1
    b.idx[::5, 2] = 64
    b.idx[::3, 3] = b.idx[::3, 0]
    b.idx[::2, 5] = b.idx[::2, 0]  # up to three times
    for fn in (0, 1, 2):
        for renorm in (True, False):
            for odt in TYPES:
                for pad in (0, 3, 8):
                    check_backward(rg, b, fn, renorm, odt, logits=strided(b.logits, pad), pad=pad)


def test_gradient_into_the_logits_themselves(rg):
    b = Batch(300, 96, 4, seed=5)
    want = torch.empty_like(b.logits)
    r = router(96, 4, 0)
    rg.route_backward(r, b.logits, dev(b.idx), want, dw=dev(b.dw))
    same = b.logits.clone()
    rg.route_backward(r, same, dev(b.idx), same, dw=dev(b.dw))
    assert torch.equal(same, want)


@pytest.mark.parametrize("fn", [0, 1, 2])
def test_gradients_against_differences(rg, fn):
    """The loss and the weights move as the gradient says: central differences of the GPU's own
    forward results, whose fp32 roundings (2^-24 of values around 1, 40 of them) over a step
    of 2^-5 leave 1e-4, and whose third derivatives (below 1) leave step^2."""
    from routed_expert_decode_gb300 import fp8

    E, k, T, step = 16, 3, 12, 2.0 ** -5
    b = Batch(T, E, k, seed=21)
    r = router(E, k, fn, s=1.0)
    ws = torch.zeros(max(rg.workspace_size(r, T), fp8.group_route_workspace_size(r, T)),
                     dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")

    def forward(l):
        idx, w = torch.empty((T, k), **i32), torch.empty((T, k), device="cuda")
        fp8.group_route(r, l, None, idx, w, torch.empty(E + 1, **i32), torch.empty(T * k, **i32),
                        torch.empty((T, k), **i32), ws)
        counts, tokens = torch.empty((1, E), **i32), torch.empty(1, **i32)
        loss = torch.empty(1, device="cuda")
        rg.balance(r, l, idx, counts, tokens, torch.empty((1, E), device="cuda"), loss, ws)
        return idx, w, counts, tokens, loss

    # picks that a step cannot change: apart by more than it
    l = b.logits.clone()
    l.scatter_add_(1, dev(b.idx).long(), 2.0 + 0.5 * torch.arange(k, device="cuda").float()
                   .expand(T, k))
    idx, w, counts, tokens, loss = forward(l)
    dw = dev(b.dw)
    g = torch.empty_like(l)
    rg.route_backward(r, l, idx, g, dw=dw, counts=counts, tokens=tokens)
    g = g.double().cpu().numpy()

    def value(l):
        i, w, _, _, loss = forward(l)
        return i, float((w.double() * dw.double()).sum()) + float(loss)

    checked = 0
    for t in range(T):
        for e in range(E):
            up, down = l.clone(), l.clone()
            up[t, e] += step
            down[t, e] -= step
            (iu, vu), (id_, vd) = value(up), value(down)
            if not (torch.equal(iu, idx) and torch.equal(id_, idx)):
                continue
            checked += 1
            assert abs((vu - vd) / (2 * step) - g[t, e]) <= 1e-4 + step ** 2, (t, e)
    assert checked > T * E // 2


# ---------------------------------------------------------------- combine's gradients
def check_combine(rg, T, k, width, R, dt, ydt, seed=0, pad=0, holes=False, dw=True, do=True):
    rng = np.random.default_rng(seed)
    o = dev(rng.standard_normal((R, width)).astype(np.float32)).to(TYPES[dt])
    dy = dev(rng.standard_normal((T, width)).astype(np.float32)).to(TYPES[ydt])
    w = rng.uniform(-1, 1, (T, k)).astype(np.float32)
    pos = rng.permutation(max(R, T * k))[:T * k].astype(np.int32).reshape(T, k)
    if holes:
        pos[rng.random((T, k)) < 0.3] = -1
    gw = torch.full((T, k), 7.0, device="cuda")
    go = torch.full((R, width + pad), 7.0, dtype=TYPES[dt], device="cuda")
    if pad:
        o, dy = strided(o, pad), strided(dy, pad)
    rg.combine_backward(dy, o, dev(w), dev(pos), gw if dw else None, go[:, :width] if do else None)
    rw, ew, ro, eo = ref.combine_backward(dy.float().cpu().numpy(), o.float().cpu().numpy(), w, pos)
    if dw:
        assert (np.abs(gw.cpu().numpy() - rw) <= ew).all()
    if do:
        got = go[:, :width].double().cpu().numpy()
        named = ~np.isnan(ro[:, 0]) if width else np.zeros(R, bool)
        bar = eo + (np.abs(ro) + eo) * HALF_ULP[dt] * (dt != "f32") + TINY[dt]
        assert (np.abs(got - ro) <= bar)[named].all()
        assert (got[~named] == 7.0).all() and (go[:, width:] == 7.0).all()


@pytest.mark.parametrize("dt,ydt", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"),
                                    ("bf16", "f32"), ("f32", "bf16"), ("f16", "bf16")])
@pytest.mark.parametrize("T,k,width", [(1, 1, 1), (1, 8, 6144), (5, 3, 257), (100, 6, 2000),
                                       (33, 32, 64), (700, 2, 1040)])
def test_combine_backward(rg, T, k, width, dt, ydt):
    check_combine(rg, T, k, width, T * k, dt, ydt)


def test_combine_backward_strides_holes_and_parts(rg):
    for pad in (0, 3, 8):
        check_combine(rg, 60, 4, 200, 260, "bf16", "bf16", pad=pad, holes=True)
        check_combine(rg, 60, 4, 200, 200, "f32", "f16", pad=pad)  # pos beyond the rows
    check_combine(rg, 20, 4, 128, 80, "bf16", "bf16", do=False)
    check_combine(rg, 20, 4, 128, 80, "bf16", "bf16", dw=False)
    check_combine(rg, 20, 4, 128, 80, "bf16", "bf16", dw=False, do=False)


def test_stream_and_graph(rg):
    """The gradients on another stream, and captured and replayed with new inputs."""
    b, b2 = Batch(200, 64, 4, 3, True, seed=1), Batch(200, 64, 4, 3, True, seed=2)
    r = router(64, 4, 0)
    ws = torch.zeros(rg.workspace_size(r, 200, 3), dtype=torch.uint8, device="cuda")
    idx, dw = dev(b.idx), dev(b.dw)
    seq, live, logits = dev(b.seq), dev(b.live), b.logits.clone()
    counts = torch.empty((3, 64), dtype=torch.int32, device="cuda")
    tokens = torch.empty(3, dtype=torch.int32, device="cuda")
    prob, loss = torch.empty((3, 64), device="cuda"), torch.empty(1, device="cuda")
    g = torch.empty_like(logits)

    def both(stream=None):
        rg.balance(r, logits, idx, counts, tokens, prob, loss, ws, seq, live, 0.5, stream)
        rg.route_backward(r, logits, idx, g, dw, counts, tokens, None, seq, live, 0.5, stream)

    def check(x):
        want, bound = ref.route_backward(
            x.l(), x.idx, 4, 0, True, 2.5, x.dw, counts.cpu().numpy(), tokens.cpu().numpy(),
            coef=0.5, **x.known())
        assert (np.abs(g.double().cpu().numpy() - want) <= bound + 1e-37).all()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    both(s)
    s.synchronize()
    check(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for x in (b2, b):
        for t, v in ((idx, x.idx), (dw, x.dw), (seq, x.seq), (live, x.live)):
            t.copy_(dev(v))
        logits.copy_(x.logits)
        graph.replay()
        check(x)


def test_beyond_32_bit_offsets(rg):
    """Logits of 8 GiB and expert rows of 12 GiB: the last tokens' results."""
    T, E, k = (1 << 22) + 3, 1024, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    tail = 40
    logits[-tail:] = torch.randn((tail, E), generator=g, device="cuda").bfloat16()
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    dw = torch.randn((T, k), generator=g, device="cuda")
    r = router(E, k, 0)
    out = torch.empty_like(logits)
    rg.route_backward(r, logits, idx, out, dw=dw)
    l, i, w = (t[-tail:].cpu().numpy() for t in (logits.float(), idx, dw))
    want, bound = ref.route_backward(l, i, k, 0, True, 2.5, w)
    bar = bound + (np.abs(want) + bound) * HALF_ULP["bf16"] + TINY["bf16"]
    assert (np.abs(out[-tail:].double().cpu().numpy() - want) <= bar).all()
    # counts of all of them, and a second sequence of the last
    seq = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")
    counts, tokens = torch.empty((2, E), dtype=torch.int32, device="cuda"), torch.empty(
        2, dtype=torch.int32, device="cuda")
    prob, loss = torch.empty((2, E), device="cuda"), torch.empty(1, device="cuda")
    ws = torch.zeros(rg.workspace_size(r, T, 2), dtype=torch.uint8, device="cuda")
    rg.balance(r, logits, idx, counts, tokens, prob, loss, ws, seq)
    n = torch.bincount(idx[:-tail].flatten().long(), minlength=E)
    assert torch.equal(counts[0].long(), n) and tokens.tolist() == [T - tail, tail]
    rc, _, rp, _, e_prob, _ = ref.balance(l, i, k, 0)
    assert np.array_equal(counts[1:].cpu().numpy(), rc)
    assert (np.abs(prob[1:].cpu().numpy() - rp) <= rp * e_prob).all()
    # equal logits: every share 1/E, each rounded as the bound of one says, summed over the
    # tokens of a CTA's warp (900 in a row) and over CTAs
    assert (prob[0] - 1.0 / E).abs().max().item() <= (70 + 900 + 700) * 2.0 ** -24 / E
    del logits, out
    R, d = (1 << 20) + 8, 6144
    o = torch.zeros((R, d), dtype=torch.bfloat16, device="cuda")
    o[-16:] = torch.randn((16, d), generator=g, device="cuda").bfloat16()
    dy = torch.randn((2, d), generator=g, device="cuda").bfloat16()
    pos = torch.arange(R - 16, R, dtype=torch.int32, device="cuda").view(2, 8)
    w = torch.rand((2, 8), generator=g, device="cuda")
    gw, go = torch.empty((2, 8), device="cuda"), torch.zeros_like(o)
    rg.combine_backward(dy, o, w, pos, gw, go)
    rw, ew, ro, eo = ref.combine_backward(dy.float().cpu().numpy(), o[-16:].float().cpu().numpy(),
                                          w.cpu().numpy(), pos.cpu().numpy() - (R - 16))
    assert (np.abs(gw.cpu().numpy() - rw) <= ew).all()
    bar = eo + (np.abs(ro) + eo) * HALF_ULP["bf16"]
    assert (np.abs(go[-16:].double().cpu().numpy() - ro) <= bar).all()
    assert not go[:-16].any()
