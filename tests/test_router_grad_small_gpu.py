"""Scores at the lower end of fp32's range: the router's gradients and its loss where the scores
of a whole token, or of all its picks, are subnormal numbers or nearly.

Bounds are router_grad_ref's.  They hold here: p adds to its 4 ulp of the exponential and two
roundings (11 units of 2^-24) two roundings to a multiple of 2^-149, 2^-22 of 2^-128 each (8
units), a sum of such p 12 more, its reciprocal and the product with it two: 19 + 31 + 2 of
the 69 units that the reference allows a share."""
import numpy as np
import pytest
import torch

from test_router_grad_gpu import Batch, check_backward, check_balance, dev, rg, router  # noqa: F401

pytestmark = pytest.mark.gpu


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
