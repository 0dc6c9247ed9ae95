"""What the fp8 operators write for one another reaches its reader in order: scales that
change from block to block and from call to call, streams, captured graphs."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from test_fp8_gpu import dev, fp8, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

ONE = 0x38  # e4m3 code of 1.0


@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("T,N", [(384, 384), (130, 128), (3000, 256)])
def test_scales_meet_their_block(fp8, T, N, gathered):  # noqa: F811
    """One product of 1 a block of K, scales of 0 or 2^kb for a row and 0 or 1 for the
    weights: an output is an integer below 2^K-blocks, exact in fp32, and names in binary
    which scales its sum took.  The scales change from call to call in place."""
    rng = np.random.default_rng(T + N)
    blocks = 20
    K = blocks * 128
    q = np.zeros((1, N, K), np.uint8)
    q[:, :, ::128] = ONE
    xq = np.zeros((T, K), np.uint8)
    xq[:, ::128] = ONE
    perm = rng.permutation(T).astype(np.int32)
    xrow = perm if gathered else np.arange(T)
    ws = workspace(fp8, T)
    wsc = torch.zeros((1, ref.nb(N), blocks), device="cuda")
    xsc = torch.zeros((T, blocks), device="cuda")
    w, x = fp8.Mat(dev(q), wsc), dev(xq)
    out = torch.empty((T, N), device="cuda")
    for _ in range(8):
        a = rng.integers(0, 2, (T, blocks)) * 2.0 ** np.arange(blocks)
        b = rng.integers(0, 2, (ref.nb(N), blocks)).astype(np.float64)
        xsc.copy_(dev(a.astype(np.float32)))
        wsc.copy_(dev(b.astype(np.float32))[None])
        out.fill_(-1)
        fp8.product(w, x, xsc, out, ws, perm=dev(perm) if gathered else None)
        want = np.repeat(a[xrow] @ b.T, 128, 1)[:, :N]
        assert np.array_equal(out.double().cpu().numpy(), want)
    assert fp8.check_device_error(ws) == 0
