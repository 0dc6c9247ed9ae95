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
