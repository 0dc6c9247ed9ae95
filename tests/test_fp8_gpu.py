"""The block-scaled fp8 operators on a GPU against the 64-bit reference.

Bars, derived from the definitions (fp8_ref): quantiser codes and scales bit for
bit; the router's picks and permutation exactly, for every token whose
selection does not rest on values closer than fp32 can tell apart; products
within their elementwise fp32 bound; h within that bound carried through SwiGLU
plus half a step of its code."""
import numpy as np
import pytest
import torch

import fp8_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


@pytest.fixture(scope="module")
def fp8(gpu):
    from routed_expert_decode_gb300 import fp8 as m

    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def strided(t, pad):
    """The same rows at a larger row stride."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


# ---------------------------------------------------------------- quantiser
def quantized(fp8, x, stream=None):
    T, d = x.shape
    q = torch.full((T, d), 0xAA, dtype=torch.uint8, device="cuda")
    s = torch.full((T, ref.nb(d)), float("nan"), device="cuda")
    fp8.quantize(x, q, s, stream)
    return q, s


def check_quantized(q, s, x):
    rq, rs, nan = ref.quantize(x.float().cpu().numpy())
    q, s = q.cpu().numpy(), s.cpu().numpy()
    assert np.array_equal(s.view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(np.isnan(ref.VALUES[q]), nan)
    assert np.array_equal(q[~nan], rq[~nan])


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,d", [(1, 1), (1, 127), (3, 128), (7, 129), (5, 1040), (2, 2000),
                                 (33, 6144), (257, 384)])
def test_quantize(fp8, dt, T, d):
    rng = np.random.default_rng(T * 1000 + d)
    x = rng.standard_normal((T, d)) * np.exp2(rng.integers(-12, 8, (T, 1)))
    x[:, rng.random(d) < 0.02] *= 50
    x = dev(x.astype(np.float32)).to(TYPES[dt])
    check_quantized(*quantized(fp8, x), x)
    x = strided(x, 13)
    check_quantized(*quantized(fp8, x), x)


def test_quantize_special_values(fp8):
    x = np.zeros((6, 256), np.float32)
    x[0] = np.linspace(-500, 500, 256)
    x[1, :] = 2.0 ** -140
    x[2, 3], x[2, 200] = np.nan, 1.0
    x[3, 7], x[3, 8], x[3, 140] = np.inf, 1.0, -np.inf
    x[4, :] = 3.0e38
    x[5, :128], x[5, 128:] = -0.0, np.nan
    x = dev(x)
    q, s = quantized(fp8, x)
    check_quantized(q, s, x)
    with np.errstate(invalid="ignore"):
        v = ref.VALUES[q.cpu().numpy()[3]] * np.repeat(s.cpu().numpy()[3], 128)
    assert np.isnan(v).all()  # an infinity leaves nothing of its block
    q, s = quantized(fp8, x[:0])
    assert q.numel() == 0


# ---------------------------------------------------------------- router
def routed(fp8, router, logits, bias, ws=None, stream=None):
    T, E = logits.shape
    k = router.top_k
    out = (torch.full((T, k), -7, dtype=torch.int32, device="cuda"),
           torch.full((T, k), float("nan"), device="cuda"),
           torch.full((E + 1,), -7, dtype=torch.int32, device="cuda"),
           torch.full((T * k,), -7, dtype=torch.int32, device="cuda"),
           torch.full((T, k), -7, dtype=torch.int32, device="cuda"))
    if ws is None:
        ws = torch.zeros(fp8.group_route_workspace_size(router, T), dtype=torch.uint8,
                         device="cuda")
    fp8.group_route(router, logits, bias, *out, ws, stream)
    assert fp8.check_device_error(ws, stream) == 0
    return [o.cpu().numpy() for o in out]


def check_routed(fp8, logits, bias, k, n_group=1, topk_group=1, score=0, top2=True, renorm=True,
                 s=2.5):
    r = fp8.make_router(logits.shape[1], k, n_group, topk_group, score, 1 if top2 else 0, renorm,
                        s)
    idx, w, off, perm, pos = routed(fp8, r, logits, bias)
    b = None if bias is None else bias.cpu().numpy()
    ridx, rw, gap = ref.route(logits.float().cpu().numpy(), b, k, n_group, topk_group, score, top2,
                              renorm, s)
    # c and the sum of two c carry a few fp32 roundings of values up to ~ 2
    sure = gap > 1e-6
    # values of c lie about 1 / E apart: few tokens have two of the k deciding ones closer
    E = logits.shape[1]
    assert (~sure).mean() <= max(0.02, 4e-6 * k * E)
    assert np.array_equal(idx[sure], ridx[sure])
    # p within 8 roundings (expf 2 ulp), the sum and the quotient a few more
    assert np.allclose(w[sure], rw[sure], rtol=32 * ref.U32, atol=1e-30)
    roff, rperm, rpos = ref.permutation(idx, logits.shape[1])
    assert np.array_equal(off, roff) and np.array_equal(perm, rperm) and np.array_equal(pos, rpos)
    return idx, w


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,E,k,G,g,score,top2,bias", [
    (1, 256, 8, 8, 4, 0, True, True),
    (5, 256, 8, 8, 4, 0, True, True),
    (32, 256, 8, 1, 1, 0, True, True),
    (33, 256, 8, 8, 2, 2, False, False),
    (300, 256, 8, 8, 4, 0, True, True),
    (1300, 64, 6, 4, 2, 2, False, False),
    (200, 160, 6, 8, 3, 2, False, False),
    (100, 384, 6, 8, 3, 0, False, True),
    (60, 384, 6, 1, 1, 1, True, True),
    (70, 96, 4, 3, 2, 0, True, False),
    (40, 21, 3, 7, 3, 0, True, True),
    (40, 1024, 32, 32, 16, 0, True, True),
    (9, 1000, 5, 4, 1, 2, True, True),
    (50, 7, 7, 1, 1, 2, False, False),
    (17, 1, 1, 1, 1, 0, True, True),
    (64, 32, 1, 32, 5, 0, True, False),
])
def test_route(fp8, dt, T, E, k, G, g, score, top2, bias):
    rng = np.random.default_rng(T + E + k)
    logits = dev(rng.standard_normal((T, E)).astype(np.float32)).to(TYPES[dt])
    b = dev((0.1 * rng.standard_normal(E)).astype(np.float32)) if bias else None
    for renorm in (True, False):
        check_routed(fp8, logits, b, k, G, g, score, top2, renorm)
    check_routed(fp8, strided(logits, 5), b, k, G, g, score, top2)


@pytest.mark.parametrize("T", [1, 31, 32, 33, 127, 1217, 20000])
def test_route_token_counts_around_the_splits(fp8, T):
    rng = np.random.default_rng(T)
    E, k = 48, 4
    r = fp8.make_router(E, k, 4, 2)
    logits = dev(rng.standard_normal((T, E)).astype(np.float32))
    idx, _, off, perm, pos = routed(fp8, r, logits, None)
    roff, rperm, rpos = ref.permutation(idx, E)
    assert np.array_equal(off, roff) and np.array_equal(perm, rperm) and np.array_equal(pos, rpos)
    n = min(T, 500)
    ridx, _, gap = ref.route(logits[:n].cpu().numpy(), None, k, 4, 2, 0, True, True, 1.0)
    assert np.array_equal(idx[:n][gap > 1e-6], ridx[gap > 1e-6])


def test_route_ties_take_the_lower_index(fp8):
    rng = np.random.default_rng(3)
    for E, G, g, k in ((256, 8, 4, 8), (160, 8, 3, 6), (40, 1, 1, 5)):
        # few distinct values: the picks rest on ties
        logits = dev(rng.integers(0, 3, (200, E)).astype(np.float32))
        check_routed(fp8, logits, None, k, G, g, 0, True)
        check_routed(fp8, logits, None, k, G, g, 2, False)
        zero = torch.zeros((3, E), device="cuda")
        idx, _ = check_routed(fp8, zero, None, k, G, g)
        assert (idx == np.arange(k)).all()


@pytest.mark.parametrize("score,top2", [(0, True), (1, True), (2, False)])
def test_route_masked_and_special_logits(fp8, score, top2):
    rng = np.random.default_rng(11)
    l = rng.standard_normal((40, 64)).astype(np.float32)
    l[0] = -np.inf                        # nothing left: the first experts, weight 0
    l[1, :60] = -np.inf                   # one group left in part
    l[2, rng.random(64) < 0.5] = np.nan   # NaN counts as -inf
    l[3] = np.finfo(np.float32).min
    l[4, [9, 33]] = np.inf
    l[5] = np.nan
    l[6, 5] = np.finfo(np.float32).min
    logits = dev(l)
    idx, w = check_routed(fp8, logits, None, 4, 8, 3, score, top2)
    assert np.isfinite(w).all()
    assert (idx[0] == np.arange(4)).all() and (idx[5] == idx[0]).all() and (w[0] == 0).all()
    if score == 2:
        assert sorted(idx[4][:2]) == [9, 33] and np.allclose(w[4][:2], 1.25)
    if score == 0:  # a bias of -inf retires experts, of the lowest value too
        b = np.zeros(64, np.float32)
        b[:16] = -np.inf
        b[16:24] = np.finfo(np.float32).min
        idx, _ = check_routed(fp8, logits[7:], dev(b), 4, 8, 3, 0, top2)
        assert (idx >= 24).all()


def test_route_agrees_with_float32_arithmetic(fp8):
    """Picks equal a float32 evaluation of the definition with torch's exp, every
    token (both call CUDA's expf), so a model that routed in torch keeps its picks."""
    rng = np.random.default_rng(5)
    logits = dev(rng.standard_normal((6000, 256)).astype(np.float32))
    bias = dev((0.1 * rng.standard_normal(256)).astype(np.float32))
    r = fp8.make_router(256, 8, 8, 4)
    idx = routed(fp8, r, logits, bias)[0]
    c = 1.0 / (1.0 + torch.exp(-logits)) + bias
    top = c.view(-1, 8, 32).topk(2, dim=2).values
    kept = (top[..., 0] + top[..., 1]).topk(4, dim=1).indices
    mask = torch.zeros((6000, 8), dtype=torch.bool, device="cuda").scatter_(1, kept, True)
    c = c.masked_fill(~mask.repeat_interleave(32, 1), -np.inf)
    want = c.sort(dim=1, descending=True, stable=True).indices[:, :8]
    assert np.array_equal(idx, want.int().cpu().numpy())


def test_route_repeats_and_shares_a_workspace(fp8):
    rng = np.random.default_rng(8)
    r = fp8.make_router(256, 8, 8, 4)
    big = dev(rng.standard_normal((3000, 256)).astype(np.float32))
    ws = torch.zeros(fp8.group_route_workspace_size(r, 3000), dtype=torch.uint8, device="cuda")
    first = routed(fp8, r, big, None, ws)
    for n in (1, 700, 3000):
        again = routed(fp8, r, big[:n], None, ws)
        assert np.array_equal(again[0], first[0][:n])
    again = routed(fp8, r, big, None, ws)
    assert all(np.array_equal(a.view(np.int32), b.view(np.int32)) for a, b in zip(first, again))
    # no tokens: the offsets alone
    off = torch.full((257,), -1, dtype=torch.int32, device="cuda")
    empty = torch.zeros((0, 8), dtype=torch.int32, device="cuda")
    fp8.group_route(r, big[:0], None, empty, empty.float(), off, empty.view(-1), empty, ws)
    assert not off.any()


# ---------------------------------------------------------------- products
def codes(rng, shape):
    v = rng.standard_normal(shape) * 100
    return ref.e4m3_encode(np.clip(v, -448, 448))


def make_mat(fp8, rng, E, N, K):
    q = codes(rng, (E, N, K))
    s = ((0.5 + rng.random((E, ref.nb(N), ref.nb(K)))) / (100 * np.sqrt(K))).astype(np.float32)
    return q, s, fp8.Mat(dev(q), dev(s))


def make_rows(rng, n, K):
    return codes(rng, (n, K)), ((0.5 + rng.random((n, ref.nb(K)))) / 100).astype(np.float32)


def assignment(rng, T, E, k, empty=()):
    """Picks of T tokens (never the experts in `empty`), and their permutation."""
    free = [e for e in range(E) if e not in empty]
    idx = np.stack([rng.choice(free, k, replace=False) for _ in range(T)]).astype(np.int32)
    return ref.permutation(idx, E)


def workspace(fp8, rows):
    return torch.zeros(fp8.workspace_size(rows), dtype=torch.uint8, device="cuda")


def expected(x, off, xrow, q, s, R, N):
    """Product of the routed rows and its bound in 64 bits; rows outside off are NaN."""
    y, e = np.full((R, N), np.nan), np.zeros((R, N))
    for i in range(len(off) - 1):
        r = slice(off[i], off[i + 1])
        if off[i + 1] > off[i]:
            y[r], e[r] = ref.product(x[xrow[r]], ref.weight(q[i], s[i]))
    return y, e


def check_out(out, y, e, dt):
    got = out.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(y))
    ok = ~np.isnan(y)
    bound = e + HALF_ULP[dt] * (np.abs(y) + e) + TINY[dt]
    worst = (np.abs(got - y)[ok] / bound[ok]).max() if ok.any() else 0.0
    assert worst <= 1.0, worst


def check_h(hq, hs, g, eg, u, eu):
    """Codes and scales of h: the scale is a's, off by no more than h's bound, and a
    code stands for h within half a step (relative 2^-4, or half of 2^-9 of the
    scale below the normal codes) of it, h's bound and the scale's error."""
    h, e = ref.swiglu(g, eg, u, eu)
    R, f = h.shape
    hs = hs.double().cpu().numpy()
    pad = np.zeros((R, ref.nb(f) * 128))
    pad[:, :f] = np.abs(h)
    epad = np.zeros_like(pad)
    epad[:, :f] = e
    a = pad.reshape(R, -1, 128).max(2)
    ea = epad.reshape(R, -1, 128).max(2)
    a = np.maximum(a, 2.0 ** -100)
    assert (np.abs(hs * 448 - a) <= ea + 4 * ref.U32 * a).all()
    v = ref.dequantize(hq.cpu().numpy(), hs)
    step = np.maximum(np.abs(h) * 2.0 ** -4, np.repeat(hs, 128, 1)[:, :f] * 2.0 ** -10)
    assert (np.abs(v - h) <= step * (1 + 2.0 ** -10) + 1.1 * e).all()


PRODUCT_CASES = [
    # T, E, k, K, N, experts without rows
    (1, 8, 2, 256, 256, ()),
    (1, 1, 1, 16, 1, ()),
    (3, 4, 2, 128, 128, (1,)),
    (5, 6, 3, 144, 136, (0, 5)),
    (33, 3, 1, 400, 264, ()),
    (70, 2, 2, 1040, 200, ()),
    (64, 40, 6, 256, 384, (3, 4, 5, 39)),
    (300, 3, 2, 512, 640, ()),
    (260, 1, 1, 2064, 520, ()),
    # 25 to 64 rows of one expert, whose tiles are split along K
    (25, 1, 1, 2064, 200, ()),
    (55, 1, 1, 1040, 300, ()),
    (128, 1, 1, 1552, 144, ()),
    (2, 1024, 8, 128, 128, ()),
    # a reduction length that tensor copies cannot take
    (5, 3, 2, 100, 130, ()),
    (40, 2, 1, 259, 33, ()),
    (1, 1, 1, 1, 1, ()),
]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,E,k,K,N,empty", PRODUCT_CASES)
def test_product(fp8, dt, T, E, k, K, N, empty):
    rng = np.random.default_rng(T * 7 + E + K + N)
    off, perm, _ = assignment(rng, T, E, k, empty)
    q, s, w = make_mat(fp8, rng, E, N, K)
    R = T * k
    ws = workspace(fp8, R)
    for gathered in (True, False):
        xq, xs = make_rows(rng, T if gathered else R, K)
        xrow = perm // k if gathered else np.arange(R)
        y, e = expected(ref.dequantize(xq, xs), off, xrow, q, s, R, N)
        for pad in (0, 3):
            out = torch.empty((R, N + pad), dtype=TYPES[dt], device="cuda")[:, :N]
            args = dict(off=dev(off), perm=dev(perm) if gathered else None, top_k=k)
            fp8.product(w, dev(xq), dev(xs), out, ws, **args)
            check_out(out, y, e, dt)
            again = torch.empty_like(out)
            fp8.product(w, dev(xq), dev(xs), again, ws, **args)
            assert torch.equal(out, again)
        if E == 1:
            out = torch.empty((R, N), dtype=TYPES[dt], device="cuda")
            fp8.product(w, dev(xq), dev(xs), out, ws, perm=dev(perm) if gathered else None,
                        top_k=k)
            check_out(out, y, e, dt)
    assert fp8.check_device_error(ws) == 0


@pytest.mark.parametrize("T,E,k,K,N,empty", PRODUCT_CASES)
def test_swiglu(fp8, T, E, k, K, N, empty):
    rng = np.random.default_rng(T * 11 + E + K + N)
    off, perm, _ = assignment(rng, T, E, k, empty)
    gq, gsc, gate = make_mat(fp8, rng, E, N, K)
    uq, usc, up = make_mat(fp8, rng, E, N, K)
    R = T * k
    ws = workspace(fp8, R)
    xq, xs = make_rows(rng, T, K)
    xs *= 3  # gates of a few units
    x = ref.dequantize(xq, xs)
    g, eg = expected(x, off, perm // k, gq, gsc, R, N)
    u, eu = expected(x, off, perm // k, uq, usc, R, N)
    outs = []
    for _ in range(2):
        hq = torch.full((R, N), 0x55, dtype=torch.uint8, device="cuda")
        hs = torch.full((R, ref.nb(N)), float("nan"), device="cuda")
        fp8.swiglu(gate, up, dev(xq), dev(xs), hq, hs, ws, off=dev(off), perm=dev(perm), top_k=k)
        outs.append((hq, hs))
    assert fp8.check_device_error(ws) == 0
    check_h(*outs[0], g, eg, u, eu)
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


# tiles of 128 rows whose last round is shared along K by pairs of CTAs: K of 40 blocks and
# more, from the last block short to a few tiles more than the 152 of a whole round
@pytest.mark.parametrize("T,E,k,K,N,empty", [
    (300, 1, 1, 5120, 256, ()),
    (130, 1, 1, 5136, 330, ()),
    (310, 3, 2, 5232, 130, ()),
    (2500, 1, 1, 5136, 2048, ()),
])
def test_product_and_swiglu_in_halves_of_a_tile(fp8, T, E, k, K, N, empty):
    test_product(fp8, "bf16", T, E, k, K, N, empty)
    if N < 2048:
        test_swiglu(fp8, T, E, k, K, N, empty)


def test_product_planes_off_their_alignment(fp8):
    """Code planes that start off a 16-byte boundary give the aligned planes' values."""
    rng = np.random.default_rng(2)
    T, E, k, K, N = 20, 4, 2, 256, 160
    off, perm, _ = assignment(rng, T, E, k)
    q, s, w = make_mat(fp8, rng, E, N, K)
    xq, xs = make_rows(rng, T, K)
    y, e = expected(ref.dequantize(xq, xs), off, perm // k, q, s, T * k, N)
    ws = workspace(fp8, T * k)

    def shifted(a):
        raw = torch.empty(a.size + 1, dtype=torch.uint8, device="cuda")
        raw[1:] = dev(a).view(-1)
        return raw[1:].view(a.shape)

    for ww, xx in ((fp8.Mat(shifted(q), dev(s)), dev(xq)), (w, shifted(xq))):
        out = torch.empty((T * k, N), device="cuda")
        fp8.product(ww, xx, dev(xs), out, ws, off=dev(off), perm=dev(perm), top_k=k)
        check_out(out, y, e, "f32")


def test_product_share_of_the_experts(fp8):
    """off + e0 with those experts' weights: the other rows are left as they are."""
    rng = np.random.default_rng(4)
    T, E, k, K, N = 50, 12, 3, 272, 144
    off, perm, _ = assignment(rng, T, E, k)
    q, s, _ = make_mat(fp8, rng, E, N, K)
    xq, xs = make_rows(rng, T, K)
    ws = workspace(fp8, T * k)
    for e0, e1 in ((0, 5), (5, 12), (7, 8)):
        sub = off[e0:e1 + 1]
        full = np.zeros(E + 1, np.int32)
        y, e = expected(ref.dequantize(xq, xs), sub, perm // k, q[e0:e1], s[e0:e1], T * k, N)
        out = torch.full((T * k, N), float("nan"), device="cuda")
        fp8.product(fp8.Mat(dev(q[e0:e1]), dev(s[e0:e1])), dev(xq), dev(xs), out, ws,
                    off=dev(off)[e0:e1 + 1], perm=dev(perm), top_k=k)
        check_out(out, y, e, "f32")
        assert fp8.check_device_error(ws) == 0


def test_product_nan_rows_stay_alone(fp8):
    """A NaN or infinite row makes its own outputs NaN, no other row's."""
    rng = np.random.default_rng(6)
    T, K, N = 40, 256, 192
    q, s, w = make_mat(fp8, rng, 1, N, K)
    x = rng.standard_normal((T, K)).astype(np.float32)
    x[3, 9], x[17, 200] = np.nan, np.inf
    xq, xs = quantized(fp8, dev(x))
    out = torch.empty((T, N), device="cuda")
    ws = workspace(fp8, T)
    fp8.product(w, xq, xs, out, ws)
    bad = torch.isnan(out).any(1).cpu().numpy()
    assert bad[3] and bad[17] and bad.sum() == 2
    assert torch.isnan(out[3]).all() and torch.isnan(out[17]).all()


def test_product_bad_routing_is_flagged(fp8):
    rng = np.random.default_rng(7)
    T, E, k, K, N = 12, 4, 2, 256, 128
    off, perm, _ = assignment(rng, T, E, k)
    _, _, w = make_mat(fp8, rng, E, N, K)
    xq, xs = make_rows(rng, T, K)
    ws = workspace(fp8, T * k)

    def call(off, perm):
        out = torch.full((T * k, N), -3.0, device="cuda")
        fp8.product(w, dev(xq), dev(xs), out, ws, off=dev(off), perm=dev(perm), top_k=k)
        return out, fp8.check_device_error(ws)

    good, st = call(off, perm)
    assert st == 0
    for i, v in ((0, -1), (2, T * k + 5), (4, 10 ** 9), (1, off[2] + 3)):
        bad = off.copy()
        bad[i] = v
        out, st = call(bad, perm)
        assert st == 6 and (out == -3.0).all()
    for v in (-1, T * k, 2 ** 31 - 1):
        bad = perm.copy()
        bad[5] = v
        out, st = call(off, bad)
        assert st == 6
        rest = np.arange(T * k) != 5
        assert torch.equal(out[rest], good[rest])
    assert torch.equal(call(off, perm)[0], good)


# ---------------------------------------------------------------- combine
@pytest.mark.parametrize("dt,ydt", [("bf16", "bf16"), ("f32", "f32"), ("f16", "f32"),
                                    ("bf16", "f16"), ("f32", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("T,k,d", [(1, 8, 6144), (3, 1, 1), (7, 3, 257), (40, 9, 264),
                                   (5, 32, 1000)])
def test_combine(fp8, dt, ydt, T, k, d):
    rng = np.random.default_rng(T + k + d)
    R = T * k
    o = dev(rng.standard_normal((R, d)).astype(np.float32)).to(TYPES[dt])
    sh = dev(rng.standard_normal((T, d)).astype(np.float32)).to(TYPES[dt])
    w = dev(rng.random((T, k)).astype(np.float32))
    pos = rng.permutation(R).astype(np.int32).reshape(T, k)
    pos[rng.random((T, k)) < 0.1] = -1  # another rank's slots
    pos[0, 0] = R                       # and one past the end
    on, wn = o.double().cpu().numpy(), w.double().cpu().numpy()
    live = (pos >= 0) & (pos < R)
    terms = np.where(live[..., None], wn[..., None] * on[np.where(live, pos, 0)], 0.0)
    for shared in (None, sh):
        base = 0.0 if shared is None else shared.double().cpu().numpy()
        y = terms.sum(1) + base
        e = (np.abs(terms).sum(1) + np.abs(base)) * (k + 2) * ref.U32
        for pad in (0, 5):
            oo, ss = (strided(o, pad), shared) if pad else (o, shared)
            out = torch.empty((T, d + pad), dtype=TYPES[ydt], device="cuda")[:, :d]
            fp8.combine(oo, w, dev(pos), out, shared=ss)
            check_out(out, y, e, ydt)


# ---------------------------------------------------------------- streams
def test_operators_on_another_stream(fp8):
    """Every operator runs on the stream it is given, and in a captured graph."""
    rng = np.random.default_rng(9)
    T, E, k, d, f = 24, 16, 4, 256, 128
    _, _, gate = make_mat(fp8, rng, E, f, d)
    _, _, up = make_mat(fp8, rng, E, f, d)
    _, _, down = make_mat(fp8, rng, E, d, f)
    r = fp8.make_router(E, k, 4, 2)
    x = dev(rng.standard_normal((T, d)).astype(np.float32))
    logits = dev(rng.standard_normal((T, E)).astype(np.float32))
    n = max(fp8.group_route_workspace_size(r, T), fp8.workspace_size(T * k))

    def buffers():
        z = lambda *shape, t=torch.float32: torch.zeros(shape, dtype=t, device="cuda")  # noqa: E731
        return dict(idx=z(T, k, t=torch.int32), w=z(T, k), off=z(E + 1, t=torch.int32),
                    perm=z(T * k, t=torch.int32), pos=z(T, k, t=torch.int32),
                    xq=z(T, d, t=torch.uint8), xs=z(T, 2), hq=z(T * k, f, t=torch.uint8),
                    hs=z(T * k, 1), o=z(T * k, d), y=z(T, d), ws=z(n, t=torch.uint8))

    def layer(b, stream):
        fp8.group_route(r, logits, None, b["idx"], b["w"], b["off"], b["perm"], b["pos"], b["ws"],
                        stream)
        fp8.quantize(x, b["xq"], b["xs"], stream)
        fp8.swiglu(gate, up, b["xq"], b["xs"], b["hq"], b["hs"], b["ws"], off=b["off"],
                   perm=b["perm"], top_k=k, stream=stream)
        fp8.product(down, b["hq"], b["hs"], b["o"], b["ws"], off=b["off"], stream=stream)
        fp8.combine(b["o"], b["w"], b["pos"], b["y"], stream=stream)

    here = buffers()
    layer(here, None)
    torch.cuda.synchronize()
    side, there = torch.cuda.Stream(), buffers()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        layer(there, side)
    side.synchronize()
    assert here["y"].abs().max() > 0 and torch.equal(here["y"], there["y"])
    third = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(third, None)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(here["y"], third["y"])
    for b in (here, there, third):
        assert fp8.check_device_error(b["ws"]) == 0


# ---------------------------------------------------------------- the layer
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,G,g,d,f,fs", [(1, 32, 4, 4, 2, 512, 256, 256),
                                              (37, 32, 4, 4, 2, 512, 272, 128),
                                              (300, 4, 2, 1, 1, 400, 256, 0)])
def test_layer_stage_by_stage(fp8, dt, T, E, k, G, g, d, f, fs):
    """fp8.Layer's every stage against the reference on that stage's own inputs."""
    rng = np.random.default_rng(T + E)
    mats = [make_mat(fp8, rng, E, f, d), make_mat(fp8, rng, E, f, d), make_mat(fp8, rng, E, d, f)]
    sh = [make_mat(fp8, rng, 1, fs, d), make_mat(fp8, rng, 1, fs, d),
          make_mat(fp8, rng, 1, d, fs)] if fs else None
    layer = fp8.Layer(fp8.make_router(E, k, G, g, s=2.5), *(m[2] for m in mats),
                      shared=tuple(m[2] for m in sh) if fs else None)
    x = dev(2 * rng.standard_normal((T, d)).astype(np.float32)).to(TYPES[dt])
    logits = dev(rng.standard_normal((T, E)).astype(np.float32)).to(TYPES[dt])
    bias = dev((0.1 * rng.standard_normal(E)).astype(np.float32))
    out = layer.forward(x, logits, bias)
    first = out.y.clone()
    assert torch.equal(layer.forward(x, logits, bias).y, first)
    assert fp8.check_device_error(layer.buffers(T, x.dtype)["ws"]) == 0
    idx = out.idx.cpu().numpy()
    ridx, rw, gap = ref.route(logits.float().cpu().numpy(), bias.cpu().numpy(), k, G, g, 0, True,
                              True, 2.5)
    assert np.array_equal(idx[gap > 1e-6], ridx[gap > 1e-6])
    off, perm, pos = ref.permutation(idx, E)
    assert np.array_equal(out.off.cpu().numpy(), off)
    check_quantized(out.xq.view(torch.uint8), out.xs, x)
    R = T * k

    def codes_of(q, s):
        return ref.dequantize(q.view(torch.uint8).cpu().numpy(), s.cpu().numpy())

    xv = codes_of(out.xq, out.xs)
    gu = [expected(xv, off, perm // k, m[0], m[1], R, f) for m in mats[:2]]
    check_h(out.hq.view(torch.uint8), out.hs, gu[0][0], gu[0][1], gu[1][0], gu[1][1])
    y, e = expected(codes_of(out.hq, out.hs), off, np.arange(R), mats[2][0], mats[2][1], R, d)
    check_out(out.o, y, e, dt)
    o = out.o.double().cpu().numpy()
    w = out.w.double().cpu().numpy()
    terms = w[..., None] * o[pos]
    base = 0.0
    if fs:
        b = layer.buffers(T, x.dtype)
        one = np.array([0, T])
        gu = [expected(xv, one, np.arange(T), m[0], m[1], T, fs) for m in sh[:2]]
        check_h(b["shq"].view(torch.uint8), b["shs"], gu[0][0], gu[0][1], gu[1][0], gu[1][1])
        y, e = expected(codes_of(b["shq"], b["shs"]), one, np.arange(T), sh[2][0], sh[2][1], T, d)
        check_out(out.shared, y, e, dt)
        base = out.shared.double().cpu().numpy()
    y = terms.sum(1) + base
    check_out(first, y, (np.abs(terms).sum(1) + np.abs(base)) * (k + 2) * ref.U32, dt)


def test_layer_example(gpu):
    """The example's layer stays near the float32 one: each of the three quantisations
    errs by at most 2^-4 of a value, independently over the hundreds that enter an
    output, so the whole stays far below 0.2 of a row's largest."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "fp8_layer.py")
    spec = importlib.util.spec_from_file_location("fp8_layer_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    for n in (1, 33, 512):
        err, _ = example.run(n)
        assert err < 0.2, err


def test_layer_refusals(fp8):
    rng = np.random.default_rng(1)
    gate, down = make_mat(fp8, rng, 4, 64, 128)[2], make_mat(fp8, rng, 4, 128, 64)[2]
    wrong = make_mat(fp8, rng, 4, 64, 112)[2]
    with pytest.raises(ValueError):
        fp8.Layer(fp8.make_router(4, 2), gate, wrong, down)
    with pytest.raises(ValueError):
        fp8.Layer(fp8.make_router(8, 2), gate, gate, down)
    with pytest.raises(ValueError):
        fp8.Layer(fp8.make_router(4, 2), gate, gate, down, shared=(gate, gate, down))
    x = torch.zeros((3, 128), device="cuda")
    out = torch.zeros((6, 128), device="cuda")
    with pytest.raises(fp8.MoeError):  # more rows asked for than there are activations
        fp8.product(down, torch.zeros((3, 64), dtype=torch.uint8, device="cuda"),
                    torch.zeros((3, 1), device="cuda"), out, workspace(fp8, 6),
                    off=torch.zeros(5, dtype=torch.int32, device="cuda"))
    with pytest.raises(fp8.MoeError):
        fp8.product(down, torch.zeros((3, 64), dtype=torch.uint8, device="cuda"),
                    torch.zeros((3, 1), device="cuda"), out[:3],
                    torch.zeros(256, dtype=torch.uint8, device="cuda"),
                    off=torch.zeros(5, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        fp8.quantize(x.double(), x, x)
    with pytest.raises(ValueError):
        fp8.quantize(x.t(), x, x)
    with pytest.raises(ValueError):
        fp8.quantize(x[:1].expand(3, 128), x, x)
