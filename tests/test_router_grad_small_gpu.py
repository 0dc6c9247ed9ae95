"""Scores at the lower end of fp32's range: the router's gradients and its loss where the scores
of a whole token, or of all its picks, are subnormal numbers, nearly or 0.

A sigmoid p below 2^-128 is 0 to the router, whose 1 + e^-l is infinite there: the reference
takes such a logit as -inf.  Bounds are router_grad_ref's.  They hold here: p adds to its 4 ulp
of the exponential and two roundings (11 units of 2^-24) two roundings to a multiple of 2^-149,
2^-22 of 2^-128 each (8 units), a sum of such p 12 more, its reciprocal and the product with it
two: 19 + 31 + 2 of the 69 units that the reference allows a share."""
import numpy as np
import pytest
import torch

from test_router_grad_gpu import Batch, check_backward, check_balance, dev, rg, router  # noqa: F401

pytestmark = pytest.mark.gpu

LEAST = np.uint32(0xC2B17217).view(np.float32)  # -88.72283: the last logit with e^-l finite


def batch(logits, k=6, dt="f32", seed=2):
    T, E = logits.shape
    b = Batch(T, E, min(E, k), 2, True, dt=dt, seed=seed)
    b.logits = dev(logits.astype(np.float32)).to(b.logits.dtype)
    return b


@pytest.mark.parametrize("fn", [0, 1])
@pytest.mark.parametrize("E", [24, 256, 384, 1000])
def test_small_coefficients_of_small_scores(rg, fn, E):  # noqa: F811
    """Products of a score and a gradient that would be subnormal where their quotient by the
    sum of the scores is not."""
    g = np.random.default_rng(E)
    for low in (-88.7, -80.0) if fn == 0 else (-168.0, -158.0):
        b = batch(g.uniform(low, low + 2, (40, E)))
        b.dw *= 1e-4
        for renorm in (True, False):
            check_backward(rg, b, fn, renorm, coef=1e-7)


@pytest.mark.parametrize("fn", [0, 1, 2])
@pytest.mark.parametrize("E", [8, 160, 512])
def test_finite_logits_have_finite_gradients(rg, fn, E):  # noqa: F811
    """Tokens of one logit, as a mask of padding leaves them, and of logits within one of it."""
    level = np.arange(-112.0, -80.0, 0.25)[:, None]
    for near in (0.0, 1.0):
        b = batch(level + near * np.random.default_rng(E).uniform(-1, 1, (len(level), E)))
        for renorm in (True, False):
            out = torch.full((b.T, E), float("nan"), device="cuda")
            counts = torch.randint(1, 9, (2, E), dtype=torch.int32, device="cuda")
            tokens = torch.full((2,), 50, dtype=torch.int32, device="cuda")
            rg.route_backward(router(E, b.k, fn, renorm), b.logits, dev(b.idx), out, dev(b.dw),
                              counts, tokens, coef=0.1, **b.where())
            assert torch.isfinite(out).all() and out.abs().max() < 1.0


class Small(Batch):
    """The reference's logits are those of the scores that the router sees."""

    def __init__(self, fn, logits, *args, **kw):
        super().__init__(*args, **kw)
        self.fn = fn
        self.logits = dev(logits.astype(np.float32)).to(self.logits.dtype)

    def l(self):
        l = super().l()
        return np.where(l < LEAST, -np.inf, l).astype(np.float32) if self.fn == 0 else l


def levels(T, E, seed):
    """Rows about one level each, from -84 to -111: a constant, a spread of one, and a wide one."""
    g = np.random.default_rng(seed)
    level = g.choice([-86.0, -87.3, -88.0, -88.6, -88.7, -89.0, -90.0, -95.0, -100.0, -103.0],
                     (T, 1))
    l = level + g.uniform(-1, 1, (T, E)) * (np.arange(T) % 3 > 0)[:, None]
    wide = np.arange(T) % 3 == 2
    l[wide] = g.uniform(-111, -84, (int(wide.sum()), E))
    return l


@pytest.mark.parametrize("fn", [0, 1, 2])
@pytest.mark.parametrize("E", [1, 24, 64, 160, 256, 384, 1000])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_small_scores(rg, fn, E, dt):  # noqa: F811
    b = Small(fn, levels(60, E, E), 60, E, min(E, 4), 2, True, dt=dt, seed=E)
    check_balance(rg, b, fn, 0.01)
    for renorm in (True, False):
        for odt in {"f32", dt}:
            check_backward(rg, b, fn, renorm, odt)
            check_backward(rg, b, fn, renorm, odt, loss=False)
            check_backward(rg, b, fn, renorm, odt, dw=False)
    b.dw[:] = 0
    check_backward(rg, b, fn, True)


@pytest.mark.parametrize("renorm", [True, False])
def test_a_masked_token_spoils_no_gradient(rg, renorm):  # noqa: F811
    """Padding rows of -100: finite rows, and zeros, as the router gives them no weight."""
    b = Batch(50, 64, 6, padded=True, seed=3)
    pad = np.flatnonzero(b.live == 0)
    b.logits[dev(pad)] = -100.0
    got = check_backward(rg, Small(0, b.logits.cpu().numpy(), 50, 64, 6, padded=True, seed=3), 0,
                         renorm)
    assert np.isfinite(got).all() and not got[pad].any()


def router_scores(fn, logits):
    """The router's own p of every expert: unnormalised weights of all of them."""
    from routed_expert_decode_gb300 import fp8

    T, E = logits.shape
    r = fp8.make_router(E, E, score=fn, renorm=False, s=1.0)
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, w = torch.empty((T, E), **i32), torch.empty((T, E), device="cuda")
    ws = torch.zeros(fp8.group_route_workspace_size(r, T), dtype=torch.uint8, device="cuda")
    fp8.group_route(r, logits, None, idx, w, torch.empty(E + 1, **i32), torch.empty(T * E, **i32),
                    torch.empty((T, E), **i32), ws)
    p = torch.empty((T, E), device="cuda").scatter_(1, idx.long(), w)
    return p.double().cpu().numpy()


def border_rows():
    l = np.random.default_rng(7).uniform(-100, -85, (40, 32)).astype(np.float32)
    bits = np.arange(0xC2B17210, 0xC2B17230, dtype=np.uint32).view(np.float32)  # about LEAST
    l[0], l[1], l[2], l[3] = bits, LEAST, np.nextafter(LEAST, np.float32(-np.inf)), -95.0
    l[4:12] = np.random.default_rng(8).uniform(-89.5, -87.0, (8, 32))
    return l


@pytest.mark.parametrize("fn", [0, 1, 2])
def test_shares_are_of_the_routers_scores(rg, fn):  # noqa: F811
    """Token by token (a sequence each).  The bar is two shares' (the loss's and the router's) and,
    for sqrt(softplus), that the router's e^l is a multiple of 2^-149, within two of them."""
    l = border_rows()
    T, E = l.shape
    p = router_scores(fn, dev(l))
    b = Batch(T, E, 4, T, seed=1)
    b.logits, b.seq = dev(l), np.arange(T + 1, dtype=np.int32)
    r = router(E, 4, fn)
    prob = torch.empty((T, E), device="cuda")
    rg.balance(r, b.logits, dev(b.idx), torch.empty((T, E), dtype=torch.int32, device="cuda"),
               torch.empty(T, dtype=torch.int32, device="cuda"), prob,
               torch.empty(1, device="cuda"),
               torch.zeros(rg.workspace_size(r, T, T), dtype=torch.uint8, device="cuda"),
               dev(b.seq))
    prob = prob.double().cpu().numpy()
    total = p.sum(1, keepdims=True)
    want = np.where(total > 0, p / np.where(total > 0, total, 1.0), 0.0)
    rel = 2 * 80 * 2.0 ** -24 + np.zeros_like(p)
    if fn == 1:
        each = 2.0 ** -149 / np.exp(l.astype(np.float64))
        rel = rel + each + each.max(1, keepdims=True)
    elif fn == 2:
        rel = rel + 2 * (l.max(1, keepdims=True) - l + 15) * 2.0 ** -24
    assert (np.abs(prob - want) <= want * rel + 2.0 ** -126).all()
    if fn == 0:
        assert ((prob == 0) == (p == 0)).all()
        # and the gradients through the loss and the weights: none of a score of 0
        counts = torch.randint(1, 9, (T, E), dtype=torch.int32, device="cuda")
        ones = torch.ones(T, dtype=torch.int32, device="cuda")
        idx = dev(np.tile(np.arange(E, dtype=np.int32), (T, 1)))
        full = router(E, E, fn, True, 1.0)
        for dw, n in ((None, counts), (torch.randn((T, E), device="cuda"), None)):
            g = torch.full((T, E), 7.0, device="cuda")
            rg.route_backward(full, b.logits, idx, g, dw, n, None if n is None else ones,
                              seq=None if n is None else dev(b.seq))
            g = g.cpu().numpy()
            assert np.isfinite(g).all() and not g[p == 0].any()
            several = (p > 0).sum(1) > 1  # of a single score the share is 1, whatever its logit
            assert (g != 0)[(p > 0) & several[:, None]].mean() > 0.9
