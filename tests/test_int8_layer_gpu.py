"""int8.Layer and its router's gradients on a GPU: every stage against the reference on that
stage's own inputs."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import fp8_ref
import int8_ref
import router_grad_ref
from test_int8_gpu import HALF_ULP, TYPES, check, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def int8(gpu):
    from routed_expert_decode_gb300 import int8 as m

    return m


def make_mat(int8, rng, E, N, K):
    q = np.clip(np.rint(rng.standard_normal((E, N, K)) * 32), -127, 127).astype(np.int8)
    s = (rng.uniform(0.5, 1.5, (E, N)) / (32 * K ** 0.5)).astype(np.float32)
    return q, s, int8.Mat(dev(q), dev(s))


def make_layer(int8, rng, E, k, G, g, d, f, fs, fn=0, renorm=True):
    mats = [make_mat(int8, rng, E, f, d), make_mat(int8, rng, E, f, d),
            make_mat(int8, rng, E, d, f)]
    sh = [make_mat(int8, rng, 1, fs, d), make_mat(int8, rng, 1, fs, d),
          make_mat(int8, rng, 1, d, fs)] if fs else None
    router = int8.make_router(E, k, G, g, score=fn, renorm=renorm, s=2.5)
    return mats, sh, int8.Layer(router, *(m[2] for m in mats),
                                shared=tuple(m[2] for m in sh) if fs else None)


def host(*tensors):
    return [t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy() for t in tensors]


def check_codes(q, s, x):
    rq, rs = int8_ref.quantize(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)


def products(q, s, off, rows, mat, N):
    """(reference, bound) of the rows of each expert."""
    q, s = host(q, s)
    y, e = np.zeros((len(rows), N)), np.zeros((len(rows), N))
    for i in range(len(off) - 1):
        r = slice(off[i], off[i + 1])
        y[r], e[r] = int8_ref.product(q[rows[r]], s[rows[r]], mat[0][i], mat[1][i])
    return y, e


def check_experts(q, s, h, hq, hs, o, off, rows, mats, dt):
    f, d = mats[0][0].shape[1:]
    gu = [products(q, s, off, rows, m, f) for m in mats[:2]]
    check(h, *fp8_ref.swiglu(gu[0][0], gu[0][1], gu[1][0], gu[1][1]), dt)
    check_codes(hq, hs, h)
    check(o, *products(hq, hs, off, np.arange(len(rows)), mats[2], d), dt)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,E,k,G,g,d,f,fs", [(1, 32, 4, 4, 2, 512, 256, 256),
                                              (37, 32, 4, 4, 2, 512, 272, 128),
                                              (300, 4, 2, 1, 1, 400, 250, 0)])
def test_layer_stage_by_stage(int8, dt, T, E, k, G, g, d, f, fs):
    rng = np.random.default_rng(T + E)
    mats, sh, layer = make_layer(int8, rng, E, k, G, g, d, f, fs)
    x = dev(2 * rng.standard_normal((T, d)).astype(np.float32)).to(TYPES[dt])
    logits = dev(rng.standard_normal((T, E)).astype(np.float32)).to(TYPES[dt])
    bias = dev((0.1 * rng.standard_normal(E)).astype(np.float32))
    out = layer.forward(x, logits, bias)
    first = out.y.clone()
    assert torch.equal(layer.forward(x, logits, bias).y, first)
    b = layer.buffers(T, x.dtype)
    assert int8.check_device_error(b["ws"]) == 0
    idx = out.idx.cpu().numpy()
    off, perm, pos = fp8_ref.permutation(idx, E)
    assert np.array_equal(out.off.cpu().numpy(), off)
    check_codes(out.xq, out.xs, x)
    check_experts(out.xq, out.xs, b["h"], out.hq, out.hs, out.o, off, perm // k, mats, dt)
    o, w = out.o.double().cpu().numpy(), out.w.double().cpu().numpy()
    terms = w[..., None] * o[pos]
    base = 0.0
    if fs:
        check_experts(out.xq, out.xs, b["sh"], b["shq"], b["shs"], out.shared, np.array([0, T]),
                      np.arange(T), sh, dt)
        base = out.shared.double().cpu().numpy()
    y = terms.sum(1) + base
    check(first, y, (np.abs(terms).sum(1) + np.abs(base)) * (k + 2) * fp8_ref.U32, dt)


@pytest.mark.parametrize("fn,renorm", [(0, True), (1, False), (2, True), (2, False)])
def test_router_gradients_of_a_layer(int8, fn, renorm):
    """dy to dlogits, through the combine, the weights and the loss."""
    rng = np.random.default_rng(3)
    T, E, k, d = 90, 32, 4, 256
    _, _, layer = make_layer(int8, rng, E, k, 4, 2, d, 128, 128, fn, renorm)
    x = dev(rng.standard_normal((T, d)).astype(np.float32)).bfloat16()
    logits = dev(rng.standard_normal((T, E)).astype(np.float32))
    dy = dev((rng.standard_normal((T, d)) / d).astype(np.float32)).bfloat16()
    seq = np.array([0, 30, 80], np.int32)
    live = (rng.random(T) > 0.2).astype(np.uint8)
    out = layer.forward(x, logits)
    do = torch.empty_like(out.o)
    got = layer.router_gradients(out, logits, dy, coef=0.05, seq=dev(seq), live=dev(live), do=do)
    hdy, ho, hw, hpos, hidx, hl = host(dy, out.o, out.w, out.pos, out.idx, logits)
    dw, edw, rdo, edo = router_grad_ref.combine_backward(hdy, ho, hw, hpos)
    assert (np.abs(got.dw.cpu().numpy() - dw) <= edw).all()
    check(do, rdo, edo, "bf16")
    counts, tokens, prob, loss, e_prob, e_loss = router_grad_ref.balance(
        hl, hidx, k, fn, 2, seq, live, 0.05)
    assert np.array_equal(got.counts.cpu().numpy(), counts)
    assert np.array_equal(got.tokens.cpu().numpy(), tokens)
    assert abs(float(got.loss) - loss) <= loss * e_loss
    want, bound = router_grad_ref.route_backward(
        hl, hidx, k, fn, renorm, 2.5, host(got.dw)[0], counts, tokens, 1.0, 2, seq, live, 0.05)
    assert (np.abs(got.dlogits.double().cpu().numpy() - want) <= bound + 2.0 ** -126).all()
    plain = layer.router_gradients(out, logits, dy)
    assert plain.loss is None and plain.counts is None
    assert torch.equal(plain.dw, got.dw)


def test_fp8_layer_has_them_too(gpu):
    from routed_expert_decode_gb300 import fp8

    g = torch.Generator(device="cuda").manual_seed(2)

    def mat(E, N, K):
        q = (torch.randn((E, N, K), generator=g, device="cuda") * 50).to(torch.float8_e4m3fn)
        return fp8.Mat(q, torch.full((E, fp8.blocks(N), fp8.blocks(K)), 1e-3, device="cuda"))

    layer = fp8.Layer(fp8.make_router(8, 2), mat(8, 128, 256), mat(8, 128, 256), mat(8, 256, 128))
    x = torch.randn((20, 256), generator=g, device="cuda").bfloat16()
    logits = torch.randn((20, 8), generator=g, device="cuda")
    out = layer.forward(x, logits)
    got = layer.router_gradients(out, logits, torch.ones_like(out.y), coef=0.1)
    dw, edw, _, _ = router_grad_ref.combine_backward(
        np.ones((20, 256)), *host(out.o, out.w, out.pos))
    assert (np.abs(got.dw.cpu().numpy() - dw) <= edw).all()
    assert torch.isfinite(got.dlogits).all() and got.dlogits.abs().sum() > 0


def test_layer_and_gradients_in_a_graph(int8):
    rng = np.random.default_rng(5)
    T, E, d = 40, 16, 256
    _, _, layer = make_layer(int8, rng, E, 2, 1, 1, d, 128, 0)
    xs = [dev(rng.standard_normal((T, d)).astype(np.float32)).bfloat16() for _ in range(2)]
    ls = [dev(rng.standard_normal((T, E)).astype(np.float32)) for _ in range(2)]
    dy = dev(rng.standard_normal((T, d)).astype(np.float32)).bfloat16()

    def both(x, l):
        out = layer.forward(x, l)
        return out.y, layer.router_gradients(out, l, dy, coef=0.1)

    want = []
    for x, l in zip(xs, ls):
        y, g = both(x, l)
        want.append((y.clone(), g.dlogits.clone(), g.loss.clone()))
    x, l = xs[0].clone(), ls[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, g = both(x, l)
    for i in (1, 0, 1):
        x.copy_(xs[i])
        l.copy_(ls[i])
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip((y, g.dlogits, g.loss), want[i]))


def test_layer_on_streams(int8):
    """Two layers on two streams at once."""
    rng = np.random.default_rng(6)
    layers = [make_layer(int8, rng, 8, 2, 1, 1, 256, 256, 128)[2] for _ in range(2)]
    x = dev(rng.standard_normal((64, 256)).astype(np.float32)).bfloat16()
    logits = dev(rng.standard_normal((64, 8)).astype(np.float32))
    want = [l.forward(x, logits).y.clone() for l in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [l.forward(x, logits, stream=s).y for l, s in zip(layers, streams)]
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_example(gpu):
    """The router's step of the example runs, and its gradient is the formulas': dW = dlogits^T x
    within the roundings of a float32 product."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "int8_router.py")
    spec = importlib.util.spec_from_file_location("int8_router_example", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    g = torch.Generator(device="cuda").manual_seed(7)
    layer = ex.make_layer(g)
    w = torch.randn((ex.E, ex.D), generator=g, device="cuda") * ex.D ** -0.5
    seq = torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda")
    x = torch.randn((50, ex.D), generator=g, device="cuda").bfloat16()
    target = torch.zeros((50, ex.D), device="cuda")
    before = w.clone()
    err, loss, dw = ex.step(layer, w, x, target, seq, coef=0.01, rate=0.5)
    assert torch.equal(w, before - 0.5 * before.norm() / dw.norm() * dw) and err > 0 and loss > 0
    # the same gradient from the layer's own buffers, in 64 bits
    logits = x.float() @ before.t()
    out = layer.forward(x, logits)
    hl, hidx, hpos, hw, ho, hy = host(logits, out.idx, out.pos, out.w, out.o, out.y)
    gdy = 2.0 * hy / len(hy)
    gw, ew, _, _ = router_grad_ref.combine_backward(gdy, ho, hw, hpos)
    counts, tokens, *_ = router_grad_ref.balance(hl, hidx, ex.TOP_K, 0, 2, [0, 20, 50], None, 0.01)
    dl, bound = router_grad_ref.route_backward(hl, hidx, ex.TOP_K, 0, True, 2.5, gw, counts, tokens,
                                               1.0, 2, [0, 20, 50], None, 0.01)
    # an error of dw moves its token's dlogits by at most 2 s of it
    bound = bound + 5.0 * ew.max(1, keepdims=True) + 2.0 ** -24 * np.abs(dl).max()
    hx = x.float().cpu().numpy().astype(np.float64)
    want = dl.T @ hx
    bar = bound.T @ np.abs(hx) + np.abs(dl).T @ np.abs(hx) * 60 * 2.0 ** -24
    assert (np.abs(dw.cpu().numpy() - want) <= bar).all()
