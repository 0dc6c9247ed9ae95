"""A routed layer of half precision whose rows between the products pass its range."""
import numpy as np
import pytest
import torch

import fp8_ref
from test_int8_gpu import dev
from test_int8_layer_gpu import check_experts, int8, make_layer  # noqa: F401

pytestmark = pytest.mark.gpu


def large(mat, factor):
    q, s, m = mat
    s *= np.float32(factor)
    m.scale.mul_(factor)


@pytest.mark.parametrize("fs", [0, 128])
def test_half_precision_rows_with_large_h(int8, fs):  # noqa: F811
    """silu(g) u above 65504, which the codes' scale holds; the layer's outputs are small."""
    rng = np.random.default_rng(1)
    T, E, k, d, f = 40, 8, 2, 256, 128
    mats, sh, layer = make_layer(int8, rng, E, k, 1, 1, d, f, fs)
    for m in mats, sh or ():
        for mat, factor in zip(m, (400.0, 400.0, 2.0 ** -14)):
            large(mat, factor)
    x = dev(rng.standard_normal((T, d)).astype(np.float32)).half()
    logits = dev(rng.standard_normal((T, E)).astype(np.float32))
    out = layer.forward(x, logits)
    b = layer.buffers(T, x.dtype)
    assert b["h"].float().abs().max() > 65504 and torch.isfinite(out.y).all()
    off, perm, pos = fp8_ref.permutation(out.idx.cpu().numpy(), E)
    check_experts(out.xq, out.xs, b["h"], out.hq, out.hs, out.o, off, perm // k, mats, "f16")
    if fs:
        check_experts(out.xq, out.xs, b["sh"], b["shq"], b["shs"], out.shared, np.array([0, T]),
                      np.arange(T), sh, "f16")
