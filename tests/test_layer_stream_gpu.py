"""moe.Layer on a stream of its own: what a call makes, it makes and clears on that stream."""
import pytest
import torch

import synth
from parity import device_layer

pytestmark = pytest.mark.gpu

SPEC = synth.LayerSpec("stream", E=64, k=4, d=512, f=256, f_shared=256, fmt=0, s=2.5,
                       zipf_beta=0.4)
SLEEP = 1 << 29  # clocks, about a quarter of a second


def fresh_layer(gpu):
    from routed_expert_decode_gb300 import moe

    l = device_layer(SPEC, gpu)
    return moe.Layer(l.n_expert, l.top_k, l.d, l.f, l.f_shared, l.routed_fmt, l.s, l.tensors, gpu,
                     l.score)


def inputs(T, gpu):
    logits, x = synth.token_inputs(SPEC, 7, T)
    return [torch.from_numpy(a).to(gpu) for a in (x, logits, synth.bias(SPEC))]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("T", [1, 9, 70])
def test_first_call_on_a_side_stream(gpu, monkeypatch, T, raw):
    from routed_expert_decode_gb300 import moe

    args = inputs(T, gpu)
    want = fresh_layer(gpu).forward(*args).y.cpu()
    layer, side = fresh_layer(gpu), torch.cuda.Stream()
    zeros, made_on = torch.zeros, []
    monkeypatch.setattr(torch, "zeros", lambda *a, **kw: (
        made_on.append(torch.cuda.current_stream().cuda_stream), zeros(*a, **kw))[1])
    with torch.cuda.stream(side):  # what the stream's memory holds
        torch.full((moe.workspace_size(layer.desc(), T),), 0x55, dtype=torch.uint8, device=gpu)
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    out = layer.forward(*args, stream=side.cuda_stream if raw else side)
    side.synchronize()
    # one token runs on a cooperative kernel, which waits for the other stream's
    # kernels to leave the GPU; the rest runs beside them
    assert T == 1 or not torch.cuda.current_stream().query()
    assert made_on == [side.cuda_stream]
    with torch.cuda.stream(side):
        assert torch.equal(out.y.cpu(), want)
        assert moe.check_device_error(layer.workspace(T, 0)) == 0
    torch.cuda.synchronize()
    assert torch.equal(layer.forward(*args).y.cpu(), want)


def test_from_x_on_a_side_stream(gpu):
    T = 9
    x, logits, bias = inputs(T, gpu)
    g = torch.Generator(device="cuda").manual_seed(3)
    w_r = torch.randn((SPEC.E, SPEC.d), generator=g, device=gpu) / SPEC.d ** 0.5
    want = fresh_layer(gpu).forward_from_x(x, w_r, bias, torch.empty_like(logits)).y.cpu()
    layer, side = fresh_layer(gpu), torch.cuda.Stream()
    out_logits = torch.empty_like(logits)
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    out = layer.forward_from_x(x, w_r, bias, out_logits, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    with torch.cuda.stream(side):
        assert torch.equal(out.y.cpu(), want)


def test_output_outlasts_its_stream(gpu):
    """A y that is dropped while its stream still has to write it is not handed out again."""
    args = inputs(9, gpu)
    layer, side = fresh_layer(gpu), torch.cuda.Stream()
    layer.forward(*args)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    out = layer.forward(*args, stream=side)
    shape, at = out.y.shape, out.y.data_ptr()
    del out
    other = [torch.zeros(shape, device=gpu) for _ in range(4)]
    assert not side.query()
    assert at not in [t.data_ptr() for t in other]
    torch.cuda.synchronize()
    assert not any(t.any() for t in other)


def test_first_call_inside_a_capture(gpu):
    """A capture only records the clearing of a workspace that it makes: a call before its
    first replay clears it for itself."""
    from routed_expert_decode_gb300 import moe

    args = inputs(9, gpu)
    want = fresh_layer(gpu).forward(*args).y.cpu()
    layer, graph = fresh_layer(gpu), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.forward(*args).y
        ws = layer.workspace(9)
    ws[:1 << 14].fill_(0x55)  # what the memory may hold
    assert torch.equal(layer.forward(*args).y.cpu(), want) and moe.check_device_error(ws) == 0
    for _ in range(2):
        y.zero_()
        graph.replay()
        assert torch.equal(y.cpu(), want)
        assert torch.equal(layer.forward(*args).y.cpu(), want)
    assert moe.check_device_error(ws) == 0
