"""Python binding of the int8 operators (C ABI in ``include/moe_int8.h``).

Argument marshalling only, as ``fp8``, whose rules on tensors, devices, streams and errors
hold here too: a bad argument raises ``MoeError`` (or ``ValueError`` for a tensor of
another device, type or shape) before anything is enqueued.

Entry points mirror the C names: ``quantize``, ``swiglu``, ``product``.  Codes are int8
with one fp32 scale per row: per token for activations, per output channel for weights.
``Layer`` runs them as one routed layer, with ``fp8``'s router and combine.
"""
from __future__ import annotations

import ctypes

import torch

from . import fp8, moe
from .fp8 import (LayerOutput, _elsewhere, _plane, _rows2d, _stream, _ws,  # noqa: F401
                  combine, group_route, group_route_workspace_size, make_router)
from .moe import MoeError, _check, _raw_stream, check_device_error  # noqa: F401

_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_u32 = ctypes.c_uint32
_int = ctypes.c_int


class Int8Mat(ctypes.Structure):
    _fields_ = [("q", _vp), ("scale", _vp)]


class Int8Rows(ctypes.Structure):
    _fields_ = [("q", _vp), ("scale", _vp), ("n", _u32), ("rows", _u32), ("off", _vp),
                ("perm", _vp), ("top_k", _u32)]


_lib = None


def lib():
    """The library with this header's signatures (loaded once; raises if absent)."""
    global _lib
    if _lib is None:
        L = fp8.lib()
        _pm, _px = ctypes.POINTER(Int8Mat), ctypes.POINTER(Int8Rows)
        L.moe_int8_quantize.restype = _int
        L.moe_int8_quantize.argtypes = [_vp, _int, _sz, _u32, _u32, _vp, _vp, _vp]
        L.moe_int8_workspace_size.restype = _sz
        L.moe_int8_workspace_size.argtypes = [_u32]
        L.moe_int8_product.restype = _int
        L.moe_int8_product.argtypes = [_pm, _u32, _u32, _u32, _px, _vp, _int, _sz, _vp, _sz, _vp]
        L.moe_int8_swiglu.restype = _int
        L.moe_int8_swiglu.argtypes = [_pm, _pm, _u32, _u32, _u32, _px, _vp, _int, _sz, _vp, _sz,
                                      _vp]
        _lib = L
    return _lib


_CODES = (torch.int8,)
_F32 = (torch.float32,)
_I32 = (torch.int32,)


# ------------------------------------------------------------------ quantiser
def quantize(x, q, scale, stream=None) -> None:
    """moe_int8_quantize: rows of ``x`` [T, d] (float32, bfloat16 or float16) to int8 codes
    ``q`` [T, d] and fp32 scales ``scale`` [T]."""
    dev = x.get_device()
    if dev < 0 or fp8._many and dev != fp8._current_device():
        return _elsewhere(dev, quantize, x, q, scale, stream)
    T, d = x.shape
    xp, dt, ld = _rows2d(x, d, "x", dev)
    st = (_lib or lib()).moe_int8_quantize(xp, dt, ld, T, d, _plane(q, _CODES, (T, d), "q", dev),
                                           _plane(scale, _F32, (T,), "scale", dev),
                                           _raw_stream(dev) if stream is None
                                           else _stream(stream, dev))
    if st:
        _check("moe_int8_quantize", st)


# ------------------------------------------------------------------ products
class Mat:
    """Weights of E experts: codes ``q`` [E, N, K] (or [N, K]: one expert) and scales
    ``scale`` [E, N] (or [N]).  Holds the tensors."""

    def __init__(self, q: torch.Tensor, scale: torch.Tensor):
        if q.dim() == 2:
            q, scale = q[None], scale[None]
        self.E, self.N, self.K = q.shape
        self.q, self.scale = q, scale
        self.dev = q.get_device()
        if self.dev < 0:
            raise ValueError(f"q must be a CUDA tensor, got one on {q.device}")
        self.c = Int8Mat(_plane(q, _CODES, q.shape, "q", self.dev),
                         _plane(scale, _F32, (self.E, self.N), "scale", self.dev))
        self.ref = ctypes.byref(self.c)


def workspace_size(rows: int) -> int:
    """Bytes of workspace that ``swiglu`` and ``product`` need for this many output rows."""
    return int(lib().moe_int8_workspace_size(rows))


def _activation(w: Mat, xq, xs, rows: int, off, perm, top_k: int, dev: int):
    n = xq.shape[0]
    if w.dev != dev:
        raise ValueError(f"the weights must be on cuda:{dev}, got cuda:{w.dev}")
    return Int8Rows(_plane(xq, _CODES, (n, w.K), "xq", dev), _plane(xs, _F32, (n,), "xs", dev), n,
                    rows, None if off is None else _plane(off, _I32, (w.E + 1,), "off", dev),
                    None if perm is None else _plane(perm, _I32, (rows,), "perm", dev), top_k)


def product(w: Mat, xq, xs, out, ws, off=None, perm=None, top_k: int = 1, stream=None) -> None:
    """moe_int8_product: ``out`` [R, N] (float32, bfloat16 or float16) = the activation rows
    times their expert's weights, transposed.  ``off`` [E + 1] gives each expert's rows
    (None: one expert, all rows); ``perm`` [R] with ``top_k`` makes row r read activation row
    perm[r] // top_k (None: row r)."""
    dev = out.get_device()
    if dev < 0 or fp8._many and dev != fp8._current_device():
        return _elsewhere(dev, product, w, xq, xs, out, ws, off, perm, top_k, stream)
    R, N = out.shape
    if N != w.N:
        raise ValueError(f"out must have {w.N} columns, got {N}")
    op, dt, ld = _rows2d(out, N, "out", dev)
    x = _activation(w, xq, xs, R, off, perm, top_k, dev)
    wsp, wsn = _ws(ws, dev)
    st = (_lib or lib()).moe_int8_product(w.ref, w.E, N, w.K, ctypes.byref(x), op, dt, ld, wsp,
                                          wsn, _raw_stream(dev) if stream is None
                                          else _stream(stream, dev))
    if st:
        _check("moe_int8_product", st)


def swiglu(gate: Mat, up: Mat, xq, xs, h, ws, off=None, perm=None, top_k: int = 1,
           stream=None) -> None:
    """moe_int8_swiglu: ``h`` [R, f] (float32, bfloat16 or float16) = silu(x Wg) * (x Wu);
    rows as in ``product``."""
    dev = h.get_device()
    if dev < 0 or fp8._many and dev != fp8._current_device():
        return _elsewhere(dev, swiglu, gate, up, xq, xs, h, ws, off, perm, top_k, stream)
    R, f = h.shape
    if (up.E, up.N, up.K, up.dev) != (gate.E, gate.N, gate.K, gate.dev):
        raise ValueError("gate and up must have the same shape and device")
    if f != gate.N:
        raise ValueError(f"h must have {gate.N} columns, got {f}")
    hp, dt, ld = _rows2d(h, f, "h", dev)
    x = _activation(gate, xq, xs, R, off, perm, top_k, dev)
    wsp, wsn = _ws(ws, dev)
    st = (_lib or lib()).moe_int8_swiglu(gate.ref, up.ref, gate.E, f, gate.K, ctypes.byref(x), hp,
                                         dt, ld, wsp, wsn, _raw_stream(dev) if stream is None
                                         else _stream(stream, dev))
    if st:
        _check("moe_int8_swiglu", st)


# ------------------------------------------------------------------ convenience
class Layer(fp8.Layer):
    """One routed layer over int8 weights on a device, as ``fp8.Layer``: group-limited routing,
    the experts' SwiGLU and down products, the always-on shared expert, the weighted combine.
    The weights are this module's ``Mat``.  Between its product and its quantiser h is held in
    x's type, of float16 in float32: silu(g) u passes 65504 where the quantiser's scale and the
    layer's outputs do not."""

    def __init__(self, router, gate, up, down, shared=None, keep_bytes: int = 4 << 30):
        if not all(isinstance(m, Mat) for m in (gate, up, down, *(shared or ()))):
            raise ValueError("the weights must be int8.Mat")
        super().__init__(router, gate, up, down, shared, keep_bytes)

    def _make(self, T: int, dtype: torch.dtype) -> dict:
        E, k, d, f, R = self.E, self.router.top_k, self.d, self.f, T * self.router.top_k
        make = self._empty
        i32, f32, i8 = torch.int32, torch.float32, torch.int8
        h = f32 if dtype is torch.float16 else dtype
        b = dict(idx=make((T, k), i32), w=make((T, k), f32), off=make((E + 1,), i32),
                 perm=make((R,), i32), pos=make((T, k), i32), xq=make((T, d), i8),
                 xs=make((T,), f32), h=make((R, f), h), hq=make((R, f), i8),
                 hs=make((R,), f32), o=make((R, d), dtype), shared=None)
        if self.shared is not None:
            fs = self.shared[0].N
            b.update(sh=make((T, fs), h), shq=make((T, fs), i8), shs=make((T,), f32),
                     shared=make((T, d), dtype))
        n = max(group_route_workspace_size(self.router, T), workspace_size(max(R, T)))
        b["ws"] = torch.zeros(n, dtype=torch.uint8, device=self.gate.q.device)
        return b

    def _experts(self, b: dict, x: torch.Tensor) -> None:
        ws = b["ws"]
        quantize(x, b["xq"], b["xs"])
        swiglu(self.gate, self.up, b["xq"], b["xs"], b["h"], ws, off=b["off"], perm=b["perm"],
               top_k=self.router.top_k)
        quantize(b["h"], b["hq"], b["hs"])
        product(self.down, b["hq"], b["hs"], b["o"], ws, off=b["off"])
        if self.shared is not None:
            sg, su, sd = self.shared
            swiglu(sg, su, b["xq"], b["xs"], b["sh"], ws)
            quantize(b["sh"], b["shq"], b["shs"])
            product(sd, b["shq"], b["shs"], b["shared"], ws)
