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


# ---------------------------------------------------------------- the layer on a stream
def make_layer(fp8, seed=0, E=8, k=2, d=2048, f=256, **kw):  # noqa: F811
    """A layer whose products of few rows are shared along K (16 blocks, few tiles)."""
    from test_fp8_gpu import make_mat

    rng = np.random.default_rng(seed)
    mats = [make_mat(fp8, rng, E, f, d)[2], make_mat(fp8, rng, E, f, d)[2],
            make_mat(fp8, rng, E, d, f)[2]]
    sh = tuple(make_mat(fp8, rng, 1, n, m)[2] for n, m in ((f, d), (f, d), (d, f)))
    return fp8.Layer(fp8.make_router(E, k, 4, 2, s=2.5), *mats, shared=sh, **kw)


def layer_inputs(T, d=2048, E=8, seed=1):
    rng = np.random.default_rng(seed + T)
    return (dev(2 * rng.standard_normal((T, d)).astype(np.float32)).bfloat16(),
            dev(rng.standard_normal((T, E)).astype(np.float32)),
            dev((0.1 * rng.standard_normal(E)).astype(np.float32)))


SLEEP = 1 << 29  # clocks, about a quarter of a second


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("T", [1, 40])
def test_layer_first_call_on_a_side_stream(fp8, monkeypatch, T, raw):  # noqa: F811
    """A first call on a stream makes and clears its buffers there, whatever the current
    stream still has to do and whatever the memory held."""
    args = layer_inputs(T)
    want = make_layer(fp8).forward(*args).y.cpu()
    layer, side = make_layer(fp8), torch.cuda.Stream()
    zeros, made_on = torch.zeros, []
    monkeypatch.setattr(torch, "zeros", lambda *a, **kw: (
        made_on.append(torch.cuda.current_stream().cuda_stream), zeros(*a, **kw))[1])
    with torch.cuda.stream(side):  # what the stream's memory holds
        torch.full((fp8.workspace_size(4 * T) + (1 << 20),), 0x55, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    out = layer.forward(*args, stream=side.cuda_stream if raw else side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()  # it is still busy
    assert made_on and set(made_on) == {side.cuda_stream}
    with torch.cuda.stream(side):
        assert torch.equal(out.y.cpu(), want)
        assert fp8.check_device_error(layer.buffers(T, args[0].dtype)["ws"]) == 0
    torch.cuda.synchronize()
    assert torch.equal(layer.forward(*args).y.cpu(), want)  # and on the current stream after it


def test_layer_output_outlasts_its_stream(fp8):  # noqa: F811
    """A y that is dropped while its stream still has to write it is not handed out again."""
    layer, side, args = make_layer(fp8), torch.cuda.Stream(), layer_inputs(40)
    layer.forward(*args)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    out = layer.forward(*args, stream=side)
    at = out.y.data_ptr()
    del out
    other = [torch.zeros((40, 2048), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    assert not side.query()
    assert at not in [t.data_ptr() for t in other]
    torch.cuda.synchronize()
    assert not any(t.any() for t in other)


def test_layer_buffers_outlast_every_stream_that_used_them(fp8):  # noqa: F811
    """Buffers of a dropped layer wait for the other streams that its calls ran on."""
    layer, side, args = make_layer(fp8), torch.cuda.Stream(), layer_inputs(300)
    layer.forward(*args)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    layer.forward(*args, stream=side)
    b = layer.buffers(300, torch.bfloat16)
    shape, at = b["o"].shape, b["o"].data_ptr()
    del layer, b
    other = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    assert not side.query()
    assert at not in [t.data_ptr() for t in other]
    torch.cuda.synchronize()


def test_layer_first_call_inside_a_capture(fp8):  # noqa: F811
    """A capture only records the clearing of buffers that it makes: calls before its first
    replay, and other captures, clear them for themselves."""
    T = 3
    args = layer_inputs(T)
    want = make_layer(fp8).forward(*args).y.cpu()
    layer = make_layer(fp8)
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        first = layer.forward(*args).y
        ws = layer.buffers(T, args[0].dtype)["ws"]
    with torch.cuda.graph(two):
        second = layer.forward(*args).y
    ws.fill_(0x55)  # what the memory may hold
    two.replay()
    assert torch.equal(second.cpu(), want) and fp8.check_device_error(ws) == 0
    ws.fill_(0x55)
    assert torch.equal(layer.forward(*args).y.cpu(), want) and fp8.check_device_error(ws) == 0
    assert layer.buffers(T, args[0].dtype)["ws"].data_ptr() == ws.data_ptr()
    for _ in range(2):
        first.zero_()
        one.replay()
        assert torch.equal(first.cpu(), want)
        assert torch.equal(layer.forward(*args).y.cpu(), want)
    assert fp8.check_device_error(ws) == 0


def test_layer_memory_is_bounded(fp8):  # noqa: F811
    """Buffers of the least recently used token counts are dropped; results, outputs in hand
    and captured graphs do not notice."""
    def size(b):
        return sum(t.numel() * t.element_size() for t in b.values() if t is not None)

    big = size(make_layer(fp8).buffers(200, torch.bfloat16))
    layer = make_layer(fp8, keep_bytes=3 * big)
    want = {T: make_layer(fp8).forward(*layer_inputs(T)).y.cpu() for T in range(190, 201)}
    args = {T: layer_inputs(T) for T in want}
    graph = torch.cuda.CUDAGraph()
    layer.forward(*args[190])
    with torch.cuda.graph(graph):
        y = layer.forward(*args[190]).y
    kept = layer.buffers(190, torch.bfloat16)
    held = layer.forward(*args[191])
    idx = held.idx.clone()
    torch.cuda.synchronize()
    for _ in range(2):
        for T in sorted(want):
            out = layer.forward(*args[T])
            assert torch.equal(out.y.cpu(), want[T])
            assert layer.buffers(T, torch.bfloat16)["o"].data_ptr() == out.o.data_ptr()
            del out
            sets = layer._buffers
            assert sum(size(b) for k, b in sets.items() if k[0] != 190) <= 3 * big
            assert set(sets) == set(layer._used_on)
        y.zero_()
        graph.replay()
        assert torch.equal(y.cpu(), want[190])
    assert layer.buffers(190, torch.bfloat16) is kept
    assert torch.equal(held.idx, idx) and torch.equal(held.y.cpu(), want[191])
    # a set larger than the limit still serves its own calls
    small = make_layer(fp8, keep_bytes=0)
    for T in (190, 191, 190):
        assert torch.equal(small.forward(*args[T]).y.cpu(), want[T])
        assert len(small._buffers) == 1
