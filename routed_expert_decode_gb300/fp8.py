"""Python binding of the block-scaled fp8 operators (C ABI in ``include/moe_fp8.h``).

Argument marshalling only, as ``moe``: every operator runs in the library's CUDA
kernels on the caller's tensors and stream, and a bad argument raises
``MoeError`` (or ``ValueError`` for a tensor of another device, type or shape)
before anything is enqueued.  A call runs on the device of its tensors, which is all of
theirs and its stream's, whether or not it is the current one.

Entry points mirror the C names: ``group_route``, ``quantize``, ``swiglu``,
``product``, ``combine``.  A row tensor may have any row stride, its columns are
consecutive.  ``Layer`` runs them together as one routed layer.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import moe
from .moe import MoeError, _capturing, _check, _raw_stream, check_device_error  # noqa: F401

BLOCK = 128
SCORE_SIGMOID = moe.SCORE_SIGMOID
SCORE_SQRT_SOFTPLUS = moe.SCORE_SQRT_SOFTPLUS
SCORE_SOFTMAX = 2
GROUP_MAX = 0
GROUP_TOP2_SUM = 1
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_u32 = ctypes.c_uint32
_int = ctypes.c_int


class MoeRouter(ctypes.Structure):
    _fields_ = [(n, _u32) for n in ("n_expert", "top_k", "n_group", "topk_group", "score",
                                    "group_score", "renorm")] + [("s", ctypes.c_float)]


class Fp8Mat(ctypes.Structure):
    _fields_ = [("q", _vp), ("scale", _vp)]


class Fp8Rows(ctypes.Structure):
    _fields_ = [("q", _vp), ("scale", _vp), ("n", _u32), ("rows", _u32), ("off", _vp),
                ("perm", _vp), ("top_k", _u32)]


_lib = None


def lib():
    """The library with this header's signatures (loaded once; raises if absent)."""
    global _lib, _many
    if _lib is None:
        _many = torch.cuda.device_count() > 1
        L = moe.lib()
        _pr, _pm, _px = (ctypes.POINTER(t) for t in (MoeRouter, Fp8Mat, Fp8Rows))
        L.moe_group_route_workspace_size.restype = _sz
        L.moe_group_route_workspace_size.argtypes = [_pr, _u32]
        L.moe_group_route.restype = _int
        L.moe_group_route.argtypes = [_pr, _vp, _int, _sz, _vp, _u32, _vp, _vp, _vp, _vp, _vp, _vp,
                                      _sz, _vp]
        L.moe_fp8_quantize.restype = _int
        L.moe_fp8_quantize.argtypes = [_vp, _int, _sz, _u32, _u32, _vp, _vp, _vp]
        L.moe_fp8_workspace_size.restype = _sz
        L.moe_fp8_workspace_size.argtypes = [_u32]
        L.moe_fp8_product.restype = _int
        L.moe_fp8_product.argtypes = [_pm, _u32, _u32, _u32, _px, _vp, _int, _sz, _vp, _sz, _vp]
        L.moe_fp8_swiglu.restype = _int
        L.moe_fp8_swiglu.argtypes = [_pm, _pm, _u32, _u32, _u32, _px, _vp, _vp, _vp, _sz, _vp]
        L.moe_fp8_combine.restype = _int
        L.moe_fp8_combine.argtypes = [_vp, _int, _sz, _u32, _vp, _vp, _u32, _u32, _u32, _vp, _sz,
                                      _vp, _int, _sz, _vp]
        _lib = L
    return _lib


def blocks(n: int) -> int:
    """Blocks of 128 that n columns take."""
    return -(-n // BLOCK)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_many = True  # whether there may be devices other than the current one (0.3 us a call)


def _elsewhere(dev: int, call, *args) -> None:
    """``call`` with device ``dev``, which is not the current one, made current: the library
    launches on the current device.  -1 is no CUDA device."""
    if dev < 0:
        raise ValueError(f"{call.__name__} needs CUDA tensors")
    with torch.cuda.device(dev):
        call(*args)


def _stream(stream, dev: int):
    """Handle of ``stream``, which must be of device ``dev``."""
    if isinstance(stream, torch.cuda.Stream) and stream.device.index != dev:
        raise ValueError(f"stream must be of cuda:{dev}, got one of {stream.device}")
    return moe._stream(stream)


def _rows2d(t: torch.Tensor, cols: int, name: str, dev: int):
    """(pointer, dtype code, row stride) of a 2-d tensor on device ``dev`` with consecutive
    columns, which number ``cols``."""
    dt = DTYPES.get(t.dtype)
    ld, step = t.stride()
    if dt is None or step != 1 or ld < cols or t.get_device() != dev:
        rows = t.shape[0]
        if t.get_device() != dev:
            raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
        if dt is None:
            raise ValueError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
        if step != 1 and cols > 1:
            raise ValueError(f"{name} must have consecutive columns")
        if ld < cols:
            if rows > 1:
                raise ValueError(f"{name}'s rows must not overlap")
            ld = cols
    return t.data_ptr(), dt, ld


def _plane(t: torch.Tensor, dtypes, shape, name: str, dev: int) -> int:
    """Pointer of a contiguous tensor on device ``dev`` of one of the dtypes and this shape."""
    if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous tensor of {dtypes[0]} and shape "
                     f"{tuple(shape)} on cuda:{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")


_CODES = (torch.float8_e4m3fn, torch.uint8)
_F32 = (torch.float32,)
_I32 = (torch.int32,)


def _ws(ws: torch.Tensor, dev: int):
    if ws.dtype is torch.uint8 and ws.is_contiguous() and ws.get_device() == dev:
        return ws.data_ptr(), ws.numel()
    raise ValueError(f"ws must be a contiguous tensor of torch.uint8 on cuda:{dev}, got {ws.dtype} "
                     f"on {ws.device}")


# ------------------------------------------------------------------ router
def make_router(n_expert: int, top_k: int, n_group: int = 1, topk_group: int = 1,
                score: int = SCORE_SIGMOID, group_score: int = GROUP_TOP2_SUM,
                renorm: bool = True, s: float = 1.0) -> MoeRouter:
    return MoeRouter(n_expert, top_k, n_group, topk_group, score, group_score, int(renorm),
                     float(s))


def group_route_workspace_size(router: MoeRouter, T: int) -> int:
    return int(lib().moe_group_route_workspace_size(ctypes.byref(router), T))


def group_route(router: MoeRouter, logits, bias: Optional[torch.Tensor], idx, w, off, perm, pos,
                ws, stream=None) -> None:
    """moe_group_route: picks and weights of ``logits`` [T, E] (float32, bfloat16 or
    float16), and the stable row permutation by expert."""
    dev = logits.get_device()
    if dev < 0 or _many and dev != _current_device():
        return _elsewhere(dev, group_route, router, logits, bias, idx, w, off, perm, pos, ws,
                          stream)
    T, E = logits.shape
    k = router.top_k
    if E != router.n_expert:
        raise ValueError(f"logits must have {router.n_expert} columns, got {E}")
    lp, dt, ld = _rows2d(logits, E, "logits", dev)
    wsp, wsn = _ws(ws, dev)
    st = (_lib or lib()).moe_group_route(
        ctypes.byref(router), lp, dt, ld,
        None if bias is None else _plane(bias, _F32, (E,), "bias", dev), T,
        _plane(idx, _I32, (T, k), "idx", dev), _plane(w, _F32, (T, k), "w", dev),
        _plane(off, _I32, (E + 1,), "off", dev), _plane(perm, _I32, (T * k,), "perm", dev),
        _plane(pos, _I32, (T, k), "pos", dev), wsp, wsn,
        _raw_stream(dev) if stream is None else _stream(stream, dev))
    if st:
        _check("moe_group_route", st)


# ------------------------------------------------------------------ quantiser
def quantize(x, q, scale, stream=None) -> None:
    """moe_fp8_quantize: rows of ``x`` [T, d] to e4m3 codes ``q`` [T, d] and fp32
    scales ``scale`` [T, ceil(d / 128)]."""
    dev = x.get_device()
    if dev < 0 or _many and dev != _current_device():
        return _elsewhere(dev, quantize, x, q, scale, stream)
    T, d = x.shape
    xp, dt, ld = _rows2d(x, d, "x", dev)
    st = (_lib or lib()).moe_fp8_quantize(xp, dt, ld, T, d, _plane(q, _CODES, (T, d), "q", dev),
                                _plane(scale, _F32, (T, blocks(d)), "scale", dev),
                                _raw_stream(dev) if stream is None else _stream(stream, dev))
    if st:
        _check("moe_fp8_quantize", st)


# ------------------------------------------------------------------ products
class Mat:
    """Weights of E experts: codes ``q`` [E, N, K] (or [N, K]: one expert) and
    scales ``scale`` [E, ceil(N / 128), ceil(K / 128)].  Holds the tensors."""

    def __init__(self, q: torch.Tensor, scale: torch.Tensor):
        if q.dim() == 2:
            q, scale = q[None], scale[None]
        self.E, self.N, self.K = q.shape
        self.q, self.scale = q, scale
        self.dev = q.get_device()
        if self.dev < 0:
            raise ValueError(f"q must be a CUDA tensor, got one on {q.device}")
        self.c = Fp8Mat(_plane(q, _CODES, q.shape, "q", self.dev),
                        _plane(scale, _F32, (self.E, blocks(self.N), blocks(self.K)), "scale",
                               self.dev))
        self.ref = ctypes.byref(self.c)


def workspace_size(rows: int) -> int:
    """Bytes of workspace that ``swiglu`` and ``product`` need for this many output rows."""
    return int(lib().moe_fp8_workspace_size(rows))


def _activation(w: Mat, xq, xs, rows: int, off, perm, top_k: int, dev: int):
    n = xq.shape[0]
    if w.dev != dev:
        raise ValueError(f"the weights must be on cuda:{dev}, got cuda:{w.dev}")
    return Fp8Rows(_plane(xq, _CODES, (n, w.K), "xq", dev),
                   _plane(xs, _F32, (n, blocks(w.K)), "xs", dev), n, rows,
                   None if off is None else _plane(off, _I32, (w.E + 1,), "off", dev),
                   None if perm is None else _plane(perm, _I32, (rows,), "perm", dev), top_k)


def product(w: Mat, xq, xs, out, ws, off=None, perm=None, top_k: int = 1, stream=None) -> None:
    """moe_fp8_product: ``out`` [R, N] = the activation rows times their expert's
    weights, transposed.  ``off`` [E + 1] gives each expert's rows (None: one
    expert, all rows); ``perm`` [R] with ``top_k`` makes row r read activation row
    perm[r] // top_k (None: row r)."""
    dev = out.get_device()
    if dev < 0 or _many and dev != _current_device():
        return _elsewhere(dev, product, w, xq, xs, out, ws, off, perm, top_k, stream)
    R, N = out.shape
    if N != w.N:
        raise ValueError(f"out must have {w.N} columns, got {N}")
    op, dt, ld = _rows2d(out, N, "out", dev)
    x = _activation(w, xq, xs, R, off, perm, top_k, dev)
    wsp, wsn = _ws(ws, dev)
    st = (_lib or lib()).moe_fp8_product(w.ref, w.E, N, w.K, ctypes.byref(x), op, dt, ld, wsp, wsn,
                               _raw_stream(dev) if stream is None else _stream(stream, dev))
    if st:
        _check("moe_fp8_product", st)


def swiglu(gate: Mat, up: Mat, xq, xs, hq, hs, ws, off=None, perm=None, top_k: int = 1,
           stream=None) -> None:
    """moe_fp8_swiglu: ``hq`` [R, f], ``hs`` [R, ceil(f / 128)] = silu(x Wg) * (x Wu),
    quantised; rows as in ``product``."""
    dev = hq.get_device()
    if dev < 0 or _many and dev != _current_device():
        return _elsewhere(dev, swiglu, gate, up, xq, xs, hq, hs, ws, off, perm, top_k, stream)
    R = hq.shape[0]
    if (up.E, up.N, up.K, up.dev) != (gate.E, gate.N, gate.K, gate.dev):
        raise ValueError("gate and up must have the same shape and device")
    x = _activation(gate, xq, xs, R, off, perm, top_k, dev)
    wsp, wsn = _ws(ws, dev)
    st = (_lib or lib()).moe_fp8_swiglu(gate.ref, up.ref, gate.E, gate.N, gate.K, ctypes.byref(x),
                              _plane(hq, _CODES, (R, gate.N), "hq", dev),
                              _plane(hs, _F32, (R, blocks(gate.N)), "hs", dev), wsp, wsn,
                              _raw_stream(dev) if stream is None else _stream(stream, dev))
    if st:
        _check("moe_fp8_swiglu", st)


# ------------------------------------------------------------------ combine
def combine(o, w, pos, y, shared=None, stream=None) -> None:
    """moe_fp8_combine: ``y`` [T, d] = ``shared`` [T, d] + sum over slots j of
    ``w`` [T, k] * ``o`` [R, d] at row ``pos`` [T, k]."""
    dev = y.get_device()
    if dev < 0 or _many and dev != _current_device():
        return _elsewhere(dev, combine, o, w, pos, y, shared, stream)
    T, d = y.shape
    R, do = o.shape
    k = pos.shape[1]
    if do != d or (shared is not None and shared.shape != (T, d)):
        raise ValueError(f"o and shared must have {d} columns, shared {T} rows")
    op, dt, ldo = _rows2d(o, d, "o", dev)
    yp, ydt, ldy = _rows2d(y, d, "y", dev)
    sp, lds = None, 0
    if shared is not None:
        sp, sdt, lds = _rows2d(shared, d, "shared", dev)
        if sdt != dt:
            raise ValueError("shared must have o's type")
    st = (_lib or lib()).moe_fp8_combine(op, dt, ldo, R, _plane(w, _F32, (T, k), "w", dev),
                               _plane(pos, _I32, (T, k), "pos", dev), T, k, d, sp, lds, yp, ydt,
                               ldy, _raw_stream(dev) if stream is None else _stream(stream, dev))
    if st:
        _check("moe_fp8_combine", st)


# ------------------------------------------------------------------ convenience
@dataclass
class LayerOutput:
    """What a layer call computed: its result and the buffers it went through (their
    values are valid until the layer's next call with as many tokens)."""
    y: torch.Tensor
    idx: torch.Tensor
    w: torch.Tensor
    off: torch.Tensor
    perm: torch.Tensor
    pos: torch.Tensor
    xq: torch.Tensor
    xs: torch.Tensor
    hq: torch.Tensor
    hs: torch.Tensor
    o: torch.Tensor
    shared: Optional[torch.Tensor]


class Layer:
    """One routed layer over fp8 weights on a device: group-limited routing, the experts'
    SwiGLU and down products, the always-on shared expert, the weighted combine.

    ``gate``, ``up`` [E, f, d] and ``down`` [E, d, f] are ``Mat``; ``shared`` is a
    triple of one-expert ``Mat`` or None.  Buffers and the workspace are kept per number
    of tokens and type, the last used up to ``keep_bytes`` in all (and those that a
    captured graph uses: its replays need them); calls that overlap need layers (or
    streams' orders) of their own.  What a call makes, it makes on its stream.
    """

    def __init__(self, router: MoeRouter, gate: Mat, up: Mat, down: Mat, shared=None,
                 keep_bytes: int = 4 << 30):
        if len({m.dev for m in (gate, up, down, *(shared or ()))}) > 1:
            raise ValueError("the weights must be on one device")
        if (gate.E, gate.N, gate.K) != (up.E, up.N, up.K) or \
                (down.E, down.N, down.K) != (gate.E, gate.K, gate.N) or \
                router.n_expert != gate.E:
            raise ValueError("gate, up [E, f, d] and down [E, d, f] must be of the router's E "
                             "experts")
        if shared is not None:
            sg, su, sd = shared
            if (sg.E, sg.K) != (1, gate.K) or (su.E, su.N, su.K) != (1, sg.N, sg.K) or \
                    (sd.E, sd.N, sd.K) != (1, gate.K, sg.N):
                raise ValueError("shared must be (gate, up, down) of one expert")
        self.router, self.gate, self.up, self.down, self.shared = router, gate, up, down, shared
        self.E, self.f, self.d = gate.E, gate.N, gate.K
        self.keep_bytes = keep_bytes
        self._buffers = {}  # the last used at the end
        self._bytes = {}    # of each set that may be dropped
        self._used_on = {}  # handles of the streams that may use each set
        self._uncleared = set()
        self._ready = None  # the last call's set and stream: as they are for another

    def buffers(self, T: int, dtype: torch.dtype) -> dict:
        """The buffers of calls of T tokens of a type, made on the current stream if new."""
        key = (T, dtype)
        here = _raw_stream(self.gate.dev)
        if self._ready == (key, here) and not _capturing():
            return self._buffers[key]
        new = key not in self._buffers
        if new:
            E, k, d, f, R = self.E, self.router.top_k, self.d, self.f, T * self.router.top_k

            def make(shape, dt):
                return torch.empty(shape, dtype=dt, device=self.gate.q.device)

            b = dict(idx=make((T, k), torch.int32), w=make((T, k), torch.float32),
                     off=make((E + 1,), torch.int32), perm=make((R,), torch.int32),
                     pos=make((T, k), torch.int32), xq=make((T, d), torch.float8_e4m3fn),
                     xs=make((T, blocks(d)), torch.float32),
                     hq=make((R, f), torch.float8_e4m3fn),
                     hs=make((R, blocks(f)), torch.float32), o=make((R, d), dtype), shared=None)
            if self.shared is not None:
                fs = self.shared[0].N
                b.update(shq=make((T, fs), torch.float8_e4m3fn),
                         shs=make((T, blocks(fs)), torch.float32), shared=make((T, d), dtype))
            n = max(group_route_workspace_size(self.router, T), workspace_size(max(R, T)))
            b["ws"] = torch.zeros(n, dtype=torch.uint8, device=self.gate.q.device)
            self._bytes[key] = sum(t.numel() * t.element_size() for t in b.values()
                                   if t is not None)
            self._used_on[key] = {here}
        else:
            b = self._buffers.pop(key)
            if here not in self._used_on[key]:
                moe._used_here(self._used_on[key], [t for t in b.values() if t is not None],
                               self.gate.q.device)
        self._buffers[key] = b
        moe._cleared(b["ws"], key, self._uncleared, new)
        if _capturing():
            self._bytes.pop(key, None)
        self._ready = None if key in self._uncleared else (key, here)
        if new:
            self._drop_unused(key)
        return b

    def _drop_unused(self, key) -> None:
        """Forget the sets that were not used for longest, down to keep_bytes (never ``key``)."""
        total = sum(self._bytes.values())
        for old in [k for k in self._buffers if k in self._bytes and k != key]:
            if total <= self.keep_bytes:
                break
            total -= self._bytes.pop(old)
            del self._buffers[old], self._used_on[old]

    def forward(self, x: torch.Tensor, logits: torch.Tensor,
                bias: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                stream=None) -> LayerOutput:
        """y [T, d] of x [T, d] and its router logits [T, E]; y has x's type unless given.  With a
        ``stream`` the whole call runs there, and what it makes belongs to it."""
        if stream is not None:
            _stream(stream, self.gate.dev)  # refuses another device's
            caller = torch.cuda.current_stream(self.gate.q.device)
            with moe._on_stream(stream, self.gate.q.device):
                out = self.forward(x, logits, bias, y)
            if y is None:  # of the stream's memory, and the caller's to read
                out.y.record_stream(caller)
            self.buffers(x.shape[0], x.dtype)
            return out
        if _many and self.gate.dev != _current_device():
            with torch.cuda.device(self.gate.dev):
                return self.forward(x, logits, bias, y)
        T = x.shape[0]
        k = self.router.top_k
        b = self.buffers(T, x.dtype)
        if y is None:
            y = torch.empty((T, self.d), dtype=x.dtype, device=x.device)
        ws = b["ws"]
        group_route(self.router, logits, bias, b["idx"], b["w"], b["off"], b["perm"], b["pos"], ws)
        quantize(x, b["xq"], b["xs"])
        swiglu(self.gate, self.up, b["xq"], b["xs"], b["hq"], b["hs"], ws, off=b["off"],
               perm=b["perm"], top_k=k)
        product(self.down, b["hq"], b["hs"], b["o"], ws, off=b["off"])
        if self.shared is not None:
            sg, su, sd = self.shared
            swiglu(sg, su, b["xq"], b["xs"], b["shq"], b["shs"], ws)
            product(sd, b["shq"], b["shs"], b["shared"], ws)
        combine(b["o"], b["w"], b["pos"], y, shared=b["shared"])
        return LayerOutput(y=y, **{n: b[n] for n in ("idx", "w", "off", "perm", "pos", "xq", "xs",
                                                     "hq", "hs", "o", "shared")})
