"""The int8 and router-gradient bindings' checks of devices and shapes, on stand-ins of
tensors: nothing is launched and no GPU is needed."""
import pytest
import torch

from routed_expert_decode_gb300 import fp8, int8, router_grad
from test_fp8_devices import Tensor, host  # noqa: F401  (a fixture)

E, K, T, D, F, S = 4, 2, 3, 256, 128, 2


@pytest.fixture
def library(host, monkeypatch):  # noqa: F811
    for m in (int8, router_grad):
        monkeypatch.setattr(m, "_lib", host)
        monkeypatch.setattr(m, "_raw_stream", lambda dev: 100 + dev)
    return host


def arguments(dev=0):
    """Every operator's arguments by name, all on one device."""
    i32, f32, u8, i8 = torch.int32, torch.float32, torch.uint8, torch.int8

    def t(shape, dtype):
        return Tensor(shape, dtype, dev)

    def mat(n, k):
        return int8.Mat(t((E, n, k), i8), t((E, n), f32))

    R = T * K
    router = fp8.make_router(E, K)
    seq, live = t((S + 1,), i32), t((T,), u8)
    return {
        (int8, "quantize"): dict(x=t((T, D), f32), q=t((T, D), i8), scale=t((T,), f32)),
        (int8, "swiglu"): dict(gate=mat(F, D), up=mat(F, D), xq=t((T, D), i8), xs=t((T,), f32),
                               h=t((R, F), f32), ws=t((1 << 20,), u8), off=t((E + 1,), i32),
                               perm=t((R,), i32), top_k=K),
        (int8, "product"): dict(w=mat(D, F), xq=t((R, F), i8), xs=t((R,), f32),
                                out=t((R, D), f32), ws=t((1 << 20,), u8), off=t((E + 1,), i32),
                                perm=t((R,), i32)),
        (router_grad, "balance"): dict(
            router=router, logits=t((T, E), f32), idx=t((T, K), i32), counts=t((S, E), i32),
            tokens=t((S,), i32), prob=t((S, E), f32), loss=t((1,), f32), ws=t((1 << 20,), u8),
            seq=seq, live=live),
        (router_grad, "route_backward"): dict(
            router=router, logits=t((T, E), f32), idx=t((T, K), i32), dlogits=t((T, E), f32),
            dw=t((T, K), f32), counts=t((S, E), i32), tokens=t((S,), i32), dloss=t((1,), f32),
            seq=seq, live=live),
        (router_grad, "combine_backward"): dict(
            dy=t((T, D), f32), o=t((R, D), f32), w=t((T, K), f32), pos=t((T, K), i32),
            dw=t((T, K), f32), do=Other((R, D), f32, dev)),
    }


class Other(Tensor):
    """A tensor of other memory than its fellows."""

    def data_ptr(self):
        return 1 << 24


NAMES = list(arguments())


def call(name, **kw):
    return getattr(name[0], name[1])(**kw)


@pytest.mark.parametrize("name", NAMES, ids=lambda n: n[1])
def test_one_tensor_of_another_device_is_refused(library, name):
    here, there = arguments(0)[name], arguments(1)[name]
    for arg, value in there.items():
        if isinstance(value, (Tensor, int8.Mat)):
            with pytest.raises(ValueError):
                call(name, **{**here, arg: value})
            with pytest.raises(ValueError):  # and one here among those over there
                call(name, **{**there, arg: here[arg]})
            if isinstance(value, Tensor):
                with pytest.raises(ValueError):  # or of the host
                    call(name, **{**here, arg: Tensor(value.shape, value.dtype, -1)})
    assert not library.calls and library.state["device"] == 0


@pytest.mark.parametrize("dev", [0, 1])
@pytest.mark.parametrize("name", NAMES, ids=lambda n: n[1])
def test_a_call_runs_on_its_tensors_device(library, name, dev):
    call(name, **arguments(dev)[name])
    (entry, device, stream), = library.calls
    assert (device, stream) == (dev, 100 + dev)
    assert library.state["device"] == 0


@pytest.mark.parametrize("name", NAMES, ids=lambda n: n[1])
def test_a_stream_of_another_device_is_refused(library, monkeypatch, name):
    class Stream:
        def __init__(self, dev):
            self.device, self.cuda_stream = torch.device("cuda", dev), 200 + dev

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    with pytest.raises(ValueError):
        call(name, **arguments(0)[name], stream=Stream(1))
    assert not library.calls
    call(name, **arguments(1)[name], stream=Stream(1))
    call(name, **arguments(0)[name], stream=300)
    assert [c[1:] for c in library.calls] == [(1, 201), (0, 300)]


@pytest.mark.parametrize("name", NAMES, ids=lambda n: n[1])
def test_a_wrong_shape_or_type_is_refused(library, name):
    """Every tensor with a row, a column or bytes too few or of a type that none takes."""
    for arg, value in arguments(0)[name].items():
        if not isinstance(value, Tensor) or arg == "ws":
            continue
        for shape, dtype in ((value.shape, torch.float64),
                             ((value.shape[0] + 1,) + tuple(value.shape[1:]), value.dtype),
                             (tuple(value.shape[:-1]) + (value.shape[-1] + 1,), value.dtype)):
            # some of these are one consistent call of another size
            consistent = {"x": 1, "xq": 1, "logits": 1, "dlogits": 0, "dy": 1, "o": 1, "seq": 0,
                          "out": 1, "h": 1, "pos": 0}.get(arg, 0)
            if consistent and shape[0] == value.shape[0] + 1:
                continue
            with pytest.raises(ValueError):
                call(name, **{**arguments(0)[name], arg: Tensor(shape, dtype, 0)})
    assert not library.calls


def test_what_goes_together(library):
    a = arguments(0)
    back = a[(router_grad, "route_backward")]
    for missing in ("counts", "tokens"):
        with pytest.raises(ValueError):
            router_grad.route_backward(**{**back, missing: None})
    with pytest.raises(ValueError):  # two sequences without their offsets
        router_grad.route_backward(**{**back, "seq": None})
    with pytest.raises(ValueError):
        router_grad.balance(**{**a[(router_grad, "balance")], "seq": None})
    combine = a[(router_grad, "combine_backward")]
    with pytest.raises(ValueError):  # do in o's memory
        router_grad.combine_backward(**{**combine, "do": combine["o"]})
    with pytest.raises(ValueError):
        router_grad.combine_backward(**{**combine, "do": Other((T * K, D), torch.bfloat16, 0)})
    mats = a[(int8, "swiglu")]
    with pytest.raises(ValueError):  # codes of the other format
        int8.Layer(fp8.make_router(E, K), mats["gate"], mats["up"],
                   fp8.Mat(Tensor((E, D, F), torch.uint8), Tensor((E, 2, 1), torch.float32)))
    assert not library.calls
