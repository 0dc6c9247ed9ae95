"""The fp8 binding's checks of devices, on stand-ins of tensors: nothing is launched and no
GPU is needed."""
import contextlib

import pytest
import torch

from routed_expert_decode_gb300 import fp8

E, K, T, D, F = 4, 2, 3, 256, 128


class Tensor:
    """What the binding asks of a tensor."""

    def __init__(self, shape, dtype, dev=0):
        self.shape, self.dtype, self.dev = torch.Size(shape), dtype, dev

    is_cuda = property(lambda self: self.dev >= 0)
    device = property(lambda self: f"cuda:{self.dev}" if self.dev >= 0 else "cpu")

    def get_device(self):
        return self.dev

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return (self.shape[1], 1)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


class Library:
    """Records which entry ran, on which device and stream."""

    def __init__(self, state):
        self.state, self.calls = state, []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, self.state["device"], args[-1]))
            return 0
        return entry


@pytest.fixture
def host(monkeypatch):
    """A host with two devices, 0 current, whose streams have the handles 100 and 101."""
    state = {"device": 0}

    @contextlib.contextmanager
    def device(dev):
        before, state["device"] = state["device"], dev
        try:
            yield
        finally:
            state["device"] = before

    library = Library(state)
    monkeypatch.setattr(fp8, "_lib", library)
    monkeypatch.setattr(fp8, "_raw_stream", lambda dev: 100 + dev)
    monkeypatch.setattr(fp8, "_current_device", lambda: state["device"], raising=False)
    monkeypatch.setattr(fp8, "_many", True, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    return library


def arguments(dev=0):
    """Every operator's arguments by name, all on one device."""
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8

    def t(shape, dtype):
        return Tensor(shape, dtype, dev)

    def mat(n, k):
        return fp8.Mat(t((E, n, k), u8), t((E, fp8.blocks(n), fp8.blocks(k)), f32))

    R = T * K
    return {
        "group_route": dict(router=fp8.make_router(E, K), logits=t((T, E), f32), bias=t((E,), f32),
                            idx=t((T, K), i32), w=t((T, K), f32), off=t((E + 1,), i32),
                            perm=t((R,), i32), pos=t((T, K), i32), ws=t((1 << 20,), u8)),
        "quantize": dict(x=t((T, D), f32), q=t((T, D), u8), scale=t((T, 2), f32)),
        "swiglu": dict(gate=mat(F, D), up=mat(F, D), xq=t((T, D), u8), xs=t((T, 2), f32),
                       hq=t((R, F), u8), hs=t((R, 1), f32), ws=t((1 << 20,), u8),
                       off=t((E + 1,), i32), perm=t((R,), i32), top_k=K),
        "product": dict(w=mat(D, F), xq=t((R, F), u8), xs=t((R, 1), f32), out=t((R, D), f32),
                        ws=t((1 << 20,), u8), off=t((E + 1,), i32), perm=t((R,), i32)),
        "combine": dict(o=t((R, D), f32), w=t((T, K), f32), pos=t((T, K), i32), y=t((T, D), f32),
                        shared=t((T, D), f32)),
    }


NAMES = ["group_route", "quantize", "swiglu", "product", "combine"]


@pytest.mark.parametrize("name", NAMES)
def test_one_tensor_of_another_device_is_refused(host, name):
    here, there = arguments(0)[name], arguments(1)[name]
    for arg, value in there.items():
        if isinstance(value, (Tensor, fp8.Mat)):
            with pytest.raises(ValueError):
                getattr(fp8, name)(**{**here, arg: value})
            with pytest.raises(ValueError):  # and one here among those over there
                getattr(fp8, name)(**{**there, arg: here[arg]})
    assert not host.calls and host.state["device"] == 0


@pytest.mark.parametrize("name", NAMES)
def test_a_tensor_of_the_host_is_refused(host, name):
    for arg, value in arguments(0)[name].items():
        if isinstance(value, Tensor):
            with pytest.raises(ValueError):
                getattr(fp8, name)(**{**arguments(0)[name], arg: Tensor(value.shape, value.dtype, -1)})
    assert not host.calls


@pytest.mark.parametrize("dev", [0, 1])
@pytest.mark.parametrize("name", NAMES)
def test_a_call_runs_on_its_tensors_device(host, name, dev):
    getattr(fp8, name)(**arguments(dev)[name])
    (entry, device, stream), = host.calls
    assert (device, stream) == (dev, 100 + dev)
    assert host.state["device"] == 0


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(host, monkeypatch, name):
    class Stream:
        def __init__(self, dev):
            self.device, self.cuda_stream = torch.device("cuda", dev), 200 + dev

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    with pytest.raises(ValueError):
        getattr(fp8, name)(**arguments(0)[name], stream=Stream(1))
    assert not host.calls
    getattr(fp8, name)(**arguments(1)[name], stream=Stream(1))
    getattr(fp8, name)(**arguments(0)[name], stream=300)
    assert [c[1:] for c in host.calls] == [(1, 201), (0, 300)]


def test_planes_of_two_devices_are_refused(host):
    q, scale = Tensor((E, F, D), torch.uint8, 0), Tensor((E, 1, 2), torch.float32, 1)
    with pytest.raises(ValueError):
        fp8.Mat(q, scale)
    with pytest.raises(ValueError):
        fp8.Mat(Tensor((E, F, D), torch.uint8, -1), Tensor((E, 1, 2), torch.float32, -1))
    a, b = arguments(0), arguments(1)
    r = fp8.make_router(E, K)
    with pytest.raises(ValueError):
        fp8.Layer(r, a["swiglu"]["gate"], a["swiglu"]["up"], b["product"]["w"])
    fp8.Layer(r, a["swiglu"]["gate"], a["swiglu"]["up"], a["product"]["w"])
