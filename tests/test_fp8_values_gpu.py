"""Values and shapes at which the fp8 products' kernels change their way: the far ends of
SwiGLU's quotient, tiles shared along K."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from test_fp8_gpu import (assignment, check_h, check_out, dev, expected, fp8,  # noqa: F401
                          make_mat, make_rows, workspace)

pytestmark = pytest.mark.gpu

ONE = 0x38  # e4m3 code of 1.0


# the few-row kernel, the many-row kernel, the one for K that tensor copies do not take
@pytest.mark.parametrize("T,K", [(3, 128), (40, 128), (130, 128), (5, 100), (70, 100)])
def test_swiglu_of_large_negative_gates(fp8, T, K):  # noqa: F811
    """g of -80 .. -88.5, where 1 + e^-g comes up to the largest floats, and u so large that h
    is far above the smallest scale: h is g / (1 + e^-g) * u as anywhere else."""
    N = 256
    gates = np.round(np.linspace(80.0, 88.0, T) * 256) / 256  # one a row, products of scales exact
    gq = np.zeros((1, N, K), np.uint8)
    gq[:, :, :2] = ONE  # g = scale_x * scale_w * (x0 + x1)
    xq = np.zeros((T, K), np.uint8)
    xq[:, 0] = ONE
    xs = gates[:, None].astype(np.float32)
    gs = np.array([[[-1.0], [-1.0078125]]], np.float32)
    us = np.array([[[1e9], [3e8]]], np.float32)
    gate, up = fp8.Mat(dev(gq), dev(gs)), fp8.Mat(dev(gq), dev(us))
    x = ref.dequantize(xq, xs)
    off = np.array([0, T])
    g, _ = expected(x, off, np.arange(T), gq, gs, T, N)
    u, _ = expected(x, off, np.arange(T), gq, us, T, N)
    eu = 2 * ref.U32 * np.abs(u)  # the product of its scales, and its use
    assert np.array_equal(g, g.astype(np.float32)) and g.min() > -88.7  # e^-g is a float
    assert (np.abs(ref.swiglu(g, 0, u, eu)[0]).max(1) > 2.0 ** -99).all()  # scales are h's own
    hq = torch.full((T, N), 0x55, dtype=torch.uint8, device="cuda")
    hs = torch.full((T, 2), float("nan"), device="cuda")
    ws = workspace(fp8, T)
    fp8.swiglu(gate, up, dev(xq), dev(xs), hq, hs, ws)
    assert fp8.check_device_error(ws) == 0
    check_h(hq, hs, g, np.zeros_like(g), u, eu)


def any_codes(rng, shape):
    """Random codes but NaN's."""
    q = rng.integers(0, 256, shape, dtype=np.uint8)
    q[(q & 0x7F) == 0x7F] &= 0xF8
    return q


SHARED_CASES = [
    # T, E, k, N, the experts that rows go to: few tiles (or few over a whole round), which are
    # shared along K.  Tiles of 32 rows by one block of columns,
    (1, 1, 1, 1000, 1),
    (5, 4, 2, 300, 4),
    (31, 2, 1, 130, 2),
    # by two,
    (12, 24, 2, 1000, 3),
    (30, 40, 1, 500, 2),
    # by two, beyond a round of whole tiles on every SM,
    (80, 160, 8, 136, 160),
    # and of 64 rows, their second half ragged, full or empty
    (55, 1, 1, 300, 1),
    (64, 1, 1, 130, 1),
    (90, 1, 1, 520, 1),
    (110, 2, 1, 264, 2),
]


@pytest.mark.parametrize("K", [2064, 6160])
@pytest.mark.parametrize("T,E,k,N,live", SHARED_CASES)
def test_product_of_few_rows_shared_along_k(fp8, T, E, k, N, live, K):  # noqa: F811
    if E * N * K > 1 << 26:
        K = 2048
    rng = np.random.default_rng(T * 13 + E + N)
    off, perm, _ = assignment(rng, T, E, k, empty=range(live, E))
    q = any_codes(rng, (E, N, K))
    s = ((0.5 + rng.random((E, ref.nb(N), ref.nb(K)))) / (100 * np.sqrt(K))).astype(np.float32)
    w, R = fp8.Mat(dev(q), dev(s)), T * k
    ws = workspace(fp8, R)
    for gathered in (True, False):
        xq = any_codes(rng, (T if gathered else R, K))
        xs = ((0.5 + rng.random((len(xq), ref.nb(K)))) / 100).astype(np.float32)
        xrow = perm // k if gathered else np.arange(R)
        y, e = expected(ref.dequantize(xq, xs), off, xrow, q, s, R, N)
        args = dict(off=dev(off), perm=dev(perm) if gathered else None, top_k=k)
        for dt, t in (("f32", torch.float32), ("bf16", torch.bfloat16)):
            outs = []
            for _ in range(2):
                out = torch.full((R, N), float("nan"), dtype=t, device="cuda")
                fp8.product(w, dev(xq), dev(xs), out, ws, **args)
                outs.append(out)
            check_out(outs[0], y, e, dt)
            assert torch.equal(*outs)
    assert fp8.check_device_error(ws) == 0
