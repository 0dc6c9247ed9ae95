"""Outputs of a routed layer's call whose buffers a later call has taken."""
import numpy as np
import pytest
import torch

from test_int8_gpu import dev
from test_int8_layer_gpu import int8, make_layer  # noqa: F401

pytestmark = pytest.mark.gpu


def test_gradients_of_an_earlier_call_are_refused(int8):  # noqa: F811
    """Two forward calls before two backward calls, as sums of gradients over batches make them."""
    rng = np.random.default_rng(2)
    d, E = 128, 8
    layer = make_layer(int8, rng, E, 2, 1, 1, d, 128, 0)[2]

    def call(T, dt=torch.bfloat16):
        x = dev(rng.standard_normal((T, d)).astype(np.float32)).to(dt)
        logits = dev(rng.standard_normal((T, E)).astype(np.float32))
        return logits, torch.randn((T, d), device="cuda"), layer.forward(x, logits)

    l1, dy1, out1 = call(20)
    want = layer.router_gradients(out1, l1, dy1).dlogits
    # buffers of another number of tokens or another type are others
    _, _, more = call(21)
    _, _, wide = call(20, torch.float32)
    assert not (out1.stale or more.stale or wide.stale)
    assert torch.equal(layer.router_gradients(out1, l1, dy1).dlogits, want)
    l2, dy2, out2 = call(20)
    assert out1.stale and not out2.stale
    with pytest.raises(ValueError, match="earlier call"):
        layer.router_gradients(out1, l1, dy1)
    layer.router_gradients(out2, l2, dy2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    layer.forward(dev(rng.standard_normal((20, d)).astype(np.float32)).bfloat16(), l1, stream=s)
    assert out2.stale


def test_outputs_of_a_dropped_set_keep_their_values(int8):  # noqa: F811
    """The buffers of a set that the layer forgets are the output's alone."""
    rng = np.random.default_rng(3)
    layer = make_layer(int8, rng, 4, 2, 1, 1, 128, 128, 0)[2]
    layer.keep_bytes = 0
    x = dev(rng.standard_normal((16, 128)).astype(np.float32)).bfloat16()
    logits, dy = dev(rng.standard_normal((16, 4)).astype(np.float32)), torch.ones_like(x)
    out = layer.forward(x, logits)
    want = layer.router_gradients(out, logits, dy).dlogits
    layer.forward(x[:7], logits[:7])   # drops the set of 16
    layer.forward(x.flip(0), logits)   # and makes another
    assert not out.stale and torch.equal(layer.router_gradients(out, logits, dy).dlogits, want)


def test_captured_calls_count_apart(int8):  # noqa: F811
    """A capture runs nothing: an earlier output keeps its values, and a captured one is of its
    graph's replays, whatever ran between."""
    rng = np.random.default_rng(4)
    d, E, T = 128, 8, 24
    layer = make_layer(int8, rng, E, 2, 1, 1, d, 128, 0)[2]
    xs = [dev(rng.standard_normal((T, d)).astype(np.float32)).bfloat16() for _ in range(2)]
    ls = [dev(rng.standard_normal((T, E)).astype(np.float32)) for _ in range(2)]
    dy = torch.randn((T, d), device="cuda")
    want = [layer.router_gradients(layer.forward(x, l), l, dy).dlogits for x, l in zip(xs, ls)]
    plain = layer.forward(xs[0], ls[0])
    forward, backward = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(forward):
        first = layer.forward(xs[0], ls[0])
        captured = layer.forward(xs[1], ls[1])
    assert first.stale and not plain.stale
    with pytest.raises(ValueError, match="earlier call"):
        layer.router_gradients(first, ls[0], dy)
    assert torch.equal(layer.router_gradients(plain, ls[0], dy).dlogits, want[0])
    layer.forward(xs[0], ls[0])
    assert plain.stale and not captured.stale
    with torch.cuda.graph(backward):
        g = layer.router_gradients(captured, ls[1], dy)
    forward.replay()
    backward.replay()
    assert torch.equal(g.dlogits, want[1])
