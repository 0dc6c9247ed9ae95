"""Python binding of what trains a router (C ABI in ``include/moe_router_grad.h``).

Argument marshalling only, as ``fp8``, whose rules on tensors, devices, streams and errors
hold here too.  Entry points mirror the C names: ``balance`` (per-expert counts, mean
probabilities and the loss that evens them out), ``route_backward`` (the logits'
gradient), ``combine_backward`` (gradients of the weighted combine).  Gradients are
plain outputs; nothing is recorded for autograd.  ``layer_gradients`` runs them behind
a layer's forward call, of ``fp8.Layer`` or ``int8.Layer``.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import fp8
from .fp8 import LayerOutput, MoeRouter, _elsewhere, _plane, _rows2d, _stream, _ws
from .moe import MoeError, _check, _raw_stream, check_device_error  # noqa: F401

_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_u32 = ctypes.c_uint32
_int = ctypes.c_int
_f32 = ctypes.c_float


class MoeTokens(ctypes.Structure):
    _fields_ = [("T", _u32), ("S", _u32), ("seq", _vp), ("live", _vp)]


_lib = None


def lib():
    """The library with this header's signatures (loaded once; raises if absent)."""
    global _lib
    if _lib is None:
        L = fp8.lib()
        _pr, _pt = ctypes.POINTER(MoeRouter), ctypes.POINTER(MoeTokens)
        L.moe_balance_workspace_size.restype = _sz
        L.moe_balance_workspace_size.argtypes = [_pr, _u32, _u32]
        L.moe_balance.restype = _int
        L.moe_balance.argtypes = [_pr, _vp, _int, _sz, _vp, _pt, _f32, _vp, _vp, _vp, _vp, _vp,
                                  _sz, _vp]
        L.moe_route_backward.restype = _int
        L.moe_route_backward.argtypes = [_pr, _vp, _int, _sz, _vp, _vp, _pt, _vp, _vp, _vp, _f32,
                                         _vp, _int, _sz, _vp]
        L.moe_combine_backward.restype = _int
        L.moe_combine_backward.argtypes = [_vp, _int, _sz, _vp, _int, _sz, _u32, _vp, _vp, _u32,
                                           _u32, _u32, _vp, _vp, _sz, _vp]
        _lib = L
    return _lib


_F32 = (torch.float32,)
_I32 = (torch.int32,)
_BYTES = (torch.uint8, torch.bool)


def _logits(router: MoeRouter, logits, name: str, dev: int):
    if logits.shape[1] != router.n_expert:
        raise ValueError(f"{name} must have {router.n_expert} columns, got {logits.shape[1]}")
    return _rows2d(logits, router.n_expert, name, dev)


def _tokens(T: int, S: int, seq, live, dev: int) -> MoeTokens:
    if seq is None and S != 1:
        raise ValueError(f"{S} sequences need seq")
    return MoeTokens(T, S, None if seq is None else _plane(seq, _I32, (S + 1,), "seq", dev),
                     None if live is None else _plane(live, _BYTES, (T,), "live", dev))


# ------------------------------------------------------------------ the loss
def workspace_size(router: MoeRouter, T: int, S: int = 1) -> int:
    """Bytes of workspace that ``balance`` needs for T tokens of S sequences."""
    return int(lib().moe_balance_workspace_size(ctypes.byref(router), T, S))


def balance(router: MoeRouter, logits, idx, counts, tokens, prob, loss, ws, seq=None, live=None,
            coef: float = 1.0, stream=None) -> None:
    """moe_balance: ``counts`` [S, E] int32, ``tokens`` [S] int32, ``prob`` [S, E] float32 and
    ``loss`` [1] float32 of ``logits`` [T, E] and the picks ``idx`` [T, k].  ``seq`` [S + 1]:
    offsets of the sequences' tokens (None: one sequence of all); ``live`` [T] uint8 or bool:
    0 marks padding (None: no padding)."""
    dev = logits.get_device()
    if dev < 0 or fp8._many and dev != fp8._current_device():
        return _elsewhere(dev, balance, router, logits, idx, counts, tokens, prob, loss, ws, seq,
                          live, coef, stream)
    T, E = logits.shape
    S = counts.shape[0]
    lp, dt, ld = _logits(router, logits, "logits", dev)
    t = _tokens(T, S, seq, live, dev)
    wsp, wsn = _ws(ws, dev)
    st = (_lib or lib()).moe_balance(
        ctypes.byref(router), lp, dt, ld, _plane(idx, _I32, (T, router.top_k), "idx", dev),
        ctypes.byref(t), coef, _plane(counts, _I32, (S, E), "counts", dev),
        _plane(tokens, _I32, (S,), "tokens", dev), _plane(prob, _F32, (S, E), "prob", dev),
        _plane(loss, _F32, (1,), "loss", dev), wsp, wsn,
        _raw_stream(dev) if stream is None else _stream(stream, dev))
    if st:
        _check("moe_balance", st)


# ------------------------------------------------------------------ gradients
def route_backward(router: MoeRouter, logits, idx, dlogits, dw=None, counts=None, tokens=None,
                   dloss=None, seq=None, live=None, coef: float = 1.0, stream=None) -> None:
    """moe_route_backward: ``dlogits`` [T, E] (float32, bfloat16 or float16) from ``dw``
    [T, k] float32, the routing weights' gradient (None: no such part), and from the loss whose
    ``counts`` and ``tokens`` ``balance`` wrote (None: no such part) with the same ``seq``,
    ``live`` and ``coef``.  ``dloss``: float32 [1], the loss's gradient (None: 1)."""
    dev = logits.get_device()
    if dev < 0 or fp8._many and dev != fp8._current_device():
        return _elsewhere(dev, route_backward, router, logits, idx, dlogits, dw, counts, tokens,
                          dloss, seq, live, coef, stream)
    T, E = logits.shape
    k = router.top_k
    lp, dt, ld = _logits(router, logits, "logits", dev)
    if dlogits.shape[0] != T:
        raise ValueError(f"dlogits must have {T} rows, got {dlogits.shape[0]}")
    dp, odt, ldd = _logits(router, dlogits, "dlogits", dev)
    if (counts is None) != (tokens is None):
        raise ValueError("counts and tokens go together")
    if counts is None:
        t, cp, np = MoeTokens(T, 1, None, None), None, None
    else:
        S = counts.shape[0]
        t = _tokens(T, S, seq, live, dev)
        cp = _plane(counts, _I32, (S, E), "counts", dev)
        np = _plane(tokens, _I32, (S,), "tokens", dev)
    st = (_lib or lib()).moe_route_backward(
        ctypes.byref(router), lp, dt, ld, _plane(idx, _I32, (T, k), "idx", dev),
        None if dw is None else _plane(dw, _F32, (T, k), "dw", dev), ctypes.byref(t), cp, np,
        None if dloss is None else _plane(dloss, _F32, (1,), "dloss", dev), coef, dp, odt, ldd,
        _raw_stream(dev) if stream is None else _stream(stream, dev))
    if st:
        _check("moe_route_backward", st)


def combine_backward(dy, o, w, pos, dw=None, do=None, stream=None) -> None:
    """moe_combine_backward: of ``fp8.combine``'s y [T, d], from its gradient ``dy`` [T, d]:
    ``dw`` [T, k] float32, the weights' gradient, and ``do`` [R, d] of o's type, the rows' (each
    None: not wanted).  ``do`` must not overlap ``o`` or ``dy``; its rows that no slot names stay
    as they are."""
    dev = dy.get_device()
    if dev < 0 or fp8._many and dev != fp8._current_device():
        return _elsewhere(dev, combine_backward, dy, o, w, pos, dw, do, stream)
    T, d = dy.shape
    R, k = o.shape[0], pos.shape[1]
    if o.shape[1] != d or (do is not None and do.shape != (R, d)):
        raise ValueError(f"o and do must have {d} columns, do {R} rows")
    yp, ydt, ldy = _rows2d(dy, d, "dy", dev)
    op, dt, ldo = _rows2d(o, d, "o", dev)
    gp, ldg = None, 0
    if do is not None:
        gp, gdt, ldg = _rows2d(do, d, "do", dev)
        if gdt != dt:
            raise ValueError("do must have o's type")
        if gp == op and R > 0:
            raise ValueError("do must not be o")
    st = (_lib or lib()).moe_combine_backward(
        yp, ydt, ldy, op, dt, ldo, R, _plane(w, _F32, (T, k), "w", dev),
        _plane(pos, _I32, (T, k), "pos", dev), T, k, d,
        None if dw is None else _plane(dw, _F32, (T, k), "dw", dev), gp, ldg,
        _raw_stream(dev) if stream is None else _stream(stream, dev))
    if st:
        _check("moe_combine_backward", st)


# ------------------------------------------------------------------ convenience
@dataclass
class RouterGradients:
    """What a backward call computed; the loss's fields are None where coef is 0."""
    dlogits: torch.Tensor
    dw: torch.Tensor
    loss: Optional[torch.Tensor]
    counts: Optional[torch.Tensor]
    tokens: Optional[torch.Tensor]
    prob: Optional[torch.Tensor]


def layer_gradients(router: MoeRouter, out: LayerOutput, logits: torch.Tensor, dy: torch.Tensor,
                    coef: float = 0.0, seq=None, live=None, dloss=None, dlogits=None,
                    do=None) -> RouterGradients:
    """The gradient of a layer's router logits [T, E] from ``dy`` [T, d], that of its output
    ``out.y``, and from the balance loss with factor ``coef`` (0: none), which is computed too.
    The experts' weights are taken as constants; ``do`` [R, d], if given, receives the gradient of
    the experts' output rows.  ``out`` whose buffers a later call has taken is refused.  Runs on
    the current stream."""
    if out.stale:
        raise ValueError("out is of an earlier call: the layer's buffers hold a later one's values")
    T, k, E = logits.shape[0], router.top_k, router.n_expert

    def make(shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=logits.device)

    if dlogits is None:
        dlogits = torch.empty_like(logits, memory_format=torch.contiguous_format)
    dw = make((T, k))
    loss = counts = tokens = prob = None
    if coef:
        S = 1 if seq is None else seq.shape[0] - 1
        loss, counts, tokens = make((1,)), make((S, E), torch.int32), make((S,), torch.int32)
        prob = make((S, E))
        ws = torch.zeros(workspace_size(router, T, S), dtype=torch.uint8, device=logits.device)
        balance(router, logits, out.idx, counts, tokens, prob, loss, ws, seq, live, coef)
    combine_backward(dy, out.o, out.w, out.pos, dw, do)
    route_backward(router, logits, out.idx, dlogits, dw, counts, tokens, dloss, seq, live, coef)
    return RouterGradients(dlogits, dw, loss, counts, tokens, prob)
