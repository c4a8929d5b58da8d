"""Binding of the calls around the expert and projection products: the
residual stream with its norms, routing by scores, and low-rank adapters
(contracts in include/qsmoe.h).

As the rest of the binding, argument marshalling only: outputs are allocated
with torch when the caller does not pass them, and a non-zero status raises
``QSMError``.  What only shows on the device (a value that is not finite) goes
to dev_status, an int32 tensor; without one it is not reported.  Import the
names from the package."""
from __future__ import annotations

import ctypes

import torch

from . import QSMError, _check, lib
from .mx4 import (Mx4Tensor, _DTYPES, _empty, _empty_mx4, _Fixed, _fp32, _handle, _matrix,
                  _status, _stream_of)

_KINDS = {"rms": 1, "layer": 2}
_MX4 = 3              # h_dtype of MXFP4


class NormC(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("eps", ctypes.c_float),
                ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class ResidualNormC(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32),
                ("h_dtype", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("gate_sigmoid", ctypes.c_int32), ("scale", ctypes.c_float),
                ("post", NormC), ("pre", NormC)]


class RouterC(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("score", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("groups_kept", ctypes.c_int32),
                ("group_best", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float), ("w_split", ctypes.c_void_p),
                ("bias", ctypes.c_void_p)]


class LoraC(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("K", ctypes.c_int32), ("N", ctypes.c_int32),
                ("a", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("ranks", ctypes.c_void_p)]


def declare(L: ctypes.CDLL) -> None:
    """Argument and result types of the entry points of library L."""
    P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    L.moe_router_split_bytes.argtypes = [i32, i32]
    L.moe_router_split_bytes.restype = ctypes.c_size_t
    L.moe_router_split.argtypes = [P, i32, i32, P, P]
    L.moe_router_split.restype = ctypes.c_int
    L.moe_route_scores.argtypes = [ctypes.POINTER(RouterC), P, i64, i32, P, P, P, P]
    L.moe_route_scores.restype = ctypes.c_int
    L.lora_add.argtypes = [ctypes.POINTER(LoraC), P, i64, i32, P, i32, P, i64, P, i64, P, P]
    L.lora_add.restype = ctypes.c_int
    L.residual_norm.argtypes = [ctypes.POINTER(ResidualNormC), i32, P, i64, P, i64, P, i64,
                                P, i64, P, i64, P, P, P]
    L.residual_norm.restype = ctypes.c_int


_lib = None


def _load():
    global _lib
    _lib = lib()
    return _lib


def _ld(t: torch.Tensor, shape, dev: int, what: str) -> int:
    """The row stride of a matrix of that shape on the device, rows contiguous."""
    if t.shape != shape or t.get_device() != dev:
        raise QSMError(f"{what} must be {list(shape)} on the same device")
    return shape[1] if t.is_contiguous() else _matrix(t, what)[3]


# ------------------------------------------------------------------- norms

class Norm(_Fixed):
    """An RMS (kind="rms") or a layer norm (kind="layer") over the columns:
    weight and bias [H] fp32 or None (1 and 0).  The contents may change, the
    attributes not be replaced."""

    def __init__(self, weight=None, bias=None, *, kind: str = "rms", eps: float = 1e-6):
        if kind not in _KINDS:
            raise QSMError('Norm: kind must be "rms" or "layer"')
        if not 0 <= eps < float("inf"):
            raise QSMError("Norm: eps must be a number from 0 on")
        for t in (weight, bias):
            if t is not None and t.dim() != 1:
                raise QSMError("Norm: weight and bias must be vectors")
        self.weight, self.bias, self.kind, self.eps = weight, bias, kind, float(eps)

    def _c(self, H: int, dev: int) -> NormC:
        for t in (self.weight, self.bias):
            _fp32(t, (H,), dev, "ResidualNorm: a norm's weight and bias")
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        return NormC(_KINDS[self.kind], self.eps, p(self.weight), p(self.bias))


class ResidualNorm(_Fixed):
    """The residual stream around a block of width H:
        x' = x + scale * gate * post(y),   h = pre(x'),
    y the output of the block before and h the input of the block after; post
    and pre a Norm or None.  sigmoid_gate: the gate passes a sigmoid first."""

    def __init__(self, H: int, pre: Norm | None = None, post: Norm | None = None,
                 scale: float = 1.0, *, sigmoid_gate: bool = False, device="cuda"):
        device = torch.device(device)
        if device.type != "cuda":
            raise QSMError("ResidualNorm: device must be a GPU")
        self.device = torch.cuda.current_device() if device.index is None else device.index
        self.H, self.pre, self.post, self.scale = H, pre, post, float(scale)
        self.sigmoid_gate = bool(sigmoid_gate)
        none = NormC(0, 0.0, None, None)
        self._norms = tuple(none if n is None else n._c(H, self.device) for n in (post, pre))
        self._forms: dict = {}  # the C struct of each combination of types

    def _form(self, key):
        form = self._forms.get(key)
        if form is None:
            x, y, g, h, gate = key
            c = ResidualNormC(self.H, x, y, g, h, gate, int(self.sigmoid_gate), self.scale,
                              *self._norms)
            form = self._forms[key] = (c, ctypes.byref(c))
        return form[1]

    def __call__(self, x: torch.Tensor, y=None, gate=None, *, x_out=None, h=None,
                 dev_status=None, stream=None):
        """Returns (x', h).
          x [T, H], y [T, H] or None (then x' is x), rows contiguous, bf16, fp16 or fp32
          gate  None, [H] (all tokens), [T, 1] (one value a token) or [T, H]
          x_out None (a new tensor; without y, x itself), or where to write x' (x itself
                is fine), of x's type
          h     None (a new tensor of x's type), a dtype or "mx4" (a new one of that type), or
                where to write it: a tensor (x or y itself is fine) or an Mx4Tensor.  Without a
                pre there is no h, and None is returned."""
        what = "ResidualNorm"
        shape, dev, xt = x.shape, self.device, _DTYPES.get(x.dtype)
        if xt is None or len(shape) != 2 or shape[1] != self.H or x.get_device() != dev:
            raise QSMError(f"{what}: x must be [T, {self.H}] bf16, fp16 or fp32 on cuda:{dev}")
        T, H = shape
        ldx = H if x.is_contiguous() else _matrix(x, what)[3]
        on = _handle(dev, stream, what)
        yp = gp = op = hp = sp = None
        yt = gt = gate_kind = ldy = ldg = ldo = ht = ldh = 0
        if y is not None:
            yt = _DTYPES.get(y.dtype)
            if yt is None:
                raise QSMError(f"{what}: y must be bf16, fp16 or fp32")
            ldy = _ld(y, shape, dev, "ResidualNorm: y")
            yp = y.data_ptr()
        if gate is not None:
            gt, gs = _DTYPES.get(gate.dtype), gate.shape
            if y is None or gt is None or gate.get_device() != dev:
                raise QSMError(f"{what}: a gate needs a y, and must be bf16, fp16 or fp32 on x's device")
            if len(gs) == 1 and gs[0] == H and gate.is_contiguous():
                gate_kind = 1
            elif len(gs) == 2 and gs[0] == T and gs[1] == 1 != H:
                gate_kind, ldg = 2, gate.stride(0)
            elif gs == shape:
                gate_kind, ldg = 1, _ld(gate, shape, dev, "ResidualNorm: gate")
            else:
                raise QSMError(f"{what}: gate must be [H], [T, 1] or [T, H]")
            gp = gate.data_ptr()
        if x_out is not None:
            if x_out.dtype != x.dtype:
                raise QSMError(f"{what}: x_out must be of x's type")
            ldo = _ld(x_out, shape, dev, "ResidualNorm: x_out")
            op = x_out.data_ptr()
        elif y is not None:
            x_out = _empty(T, H, x.dtype, stream)
            op, ldo = x_out.data_ptr(), H
        if self.pre is None:
            if h is not None:
                raise QSMError(f"{what}: without a pre there is no h")
        elif isinstance(h, torch.Tensor):
            ht = _DTYPES.get(h.dtype)
            if ht is None:
                raise QSMError(f"{what}: h must be bf16, fp16 or fp32")
            ldh = _ld(h, shape, dev, "ResidualNorm: h")
            hp = h.data_ptr()
        elif isinstance(h, Mx4Tensor) or h == "mx4":
            ht = _MX4
            if h == "mx4":
                h = _empty_mx4(T, H, dev, stream)
            elif h.rows != T or h.cols != H or h.experts != 1 or h.device != dev:
                raise QSMError(f"{what}: h has another shape or device")
            hp, sp = h.c.codes, h.c.scales
        else:
            dtype = x.dtype if h is None else h
            ht = _DTYPES.get(dtype)
            if ht is None:
                raise QSMError(f'{what}: h must be a tensor, an Mx4Tensor, bf16, fp16, fp32 or "mx4"')
            h = _empty(T, H, dtype, stream)
            hp, ldh = h.data_ptr(), H
        if op is None and hp is None:
            raise QSMError(f"{what}: neither a y nor a pre: nothing to do")
        rc = (_lib or _load()).residual_norm(
            self._form((xt, yt, gt, ht, gate_kind)), T, x.data_ptr(), ldx, yp, ldy, gp, ldg,
            op, ldo, hp, ldh, sp,
            None if dev_status is None and sp is None else _status(dev_status, dev, what), on)
        if rc:
            _check(rc, "residual_norm")
        return (x if x_out is None else x_out), h


# ------------------------------------------------------------------ routing

_SCORES = {"softmax": 0, "sigmoid": 1}


class MoERouter(_Fixed):
    """A router by scores: w_router [E, H] fp32, k experts a token.
      score   "softmax" (over all experts) or "sigmoid" (of each)
      bias    [E] fp32 or None, added to the scores for the choice, not for the weights;
              -inf closes an expert
      groups, groups_kept, group_best  equal groups of experts, how many of them stay,
              and by how many of their best experts (1 or 2) they are ranked
      renormalize, scale  the weights are divided by their sum; and multiplied
    The weights are taken as they are now (split into three bf16 parts, which is what the
    calls read); the contents of bias may change.  The attributes cannot be replaced."""

    def __init__(self, w_router: torch.Tensor, k: int, score: str = "softmax", bias=None, *,
                 groups: int = 1, groups_kept: int = 1, group_best: int = 1,
                 renormalize: bool = True, scale: float = 1.0):
        what = "MoERouter"
        if score not in _SCORES:
            raise QSMError(f'{what}: score must be "softmax" or "sigmoid"')
        if (w_router.dim() != 2 or w_router.dtype is not torch.float32
                or not w_router.is_contiguous() or w_router.get_device() < 0):
            raise QSMError(f"{what}: w_router must be a contiguous fp32 [E, H] on a GPU")
        self.E, self.H = w_router.shape
        self.k, self.score, self.bias = int(k), score, bias
        self.groups, self.groups_kept, self.group_best = int(groups), int(groups_kept), int(group_best)
        self.renormalize, self.scale = bool(renormalize), float(scale)
        self.device = w_router.get_device()
        _fp32(bias, (self.E,), self.device, f"{what}: bias")
        on = _handle(self.device, None, what)
        if (self.E < 1 or self.H < 64 or self.H % 64 or self.E > 512 or not 1 <= self.k <= min(32, self.E)
                or not 1 <= self.groups <= 32 or self.E % self.groups
                or not 1 <= self.groups_kept <= self.groups
                or not 1 <= self.group_best <= min(2, self.E // self.groups)
                or self.groups_kept * (self.E // self.groups) < self.k
                or not abs(self.scale) < float("inf")):
            raise QSMError(f"{what}: H must be a multiple of 64, E at most 512, k at most 32 and no more than "
                           "the kept groups hold, groups at most 32 dividing E, group_best 1 or 2, scale finite")
        L = lib()
        self._split = torch.empty(int(L.moe_router_split_bytes(self.E, self.H)), dtype=torch.uint8,
                                  device=w_router.device)
        _check(L.moe_router_split(w_router.data_ptr(), self.E, self.H, self._split.data_ptr(), on),
               "moe_router_split")
        self.c = RouterC(self.H, self.E, self.k, _SCORES[score], self.groups, self.groups_kept,
                         self.group_best, int(self.renormalize), self.scale, self._split.data_ptr(),
                         None if bias is None else bias.data_ptr())
        self.ref = ctypes.byref(self.c)
        self._ready = Ready(self.device)

    def route(self, x, topk_idx=None, topk_w=None, dev_status=None, stream=None):
        """moe_route_scores(x, self, ...)."""
        return moe_route_scores(x, self, topk_idx, topk_w, dev_status, stream)


class Ready:
    """What an object's constructor has enqueued on the stream that was the
    current one: the first call on another stream waits for it.  A stream that
    is being captured cannot wait for what came before the capture: there the
    caller does it, with a call or a wait before the capture."""

    def __init__(self, device: int):
        self.streams = {_stream_of(device)}
        self.event = None
        if not torch.cuda.is_current_stream_capturing():
            self.event = torch.cuda.Event()
            self.event.record()

    def wait(self, on: int, stream) -> None:
        if self.event is not None and not torch.cuda.is_current_stream_capturing():
            (torch.cuda.current_stream() if stream is None else stream).wait_event(self.event)
            self.streams.add(on)


def moe_route_scores(x: torch.Tensor, router: MoERouter, topk_idx=None, topk_w=None,
                     dev_status=None, stream=None):
    """The router's choice for x [T, H] bf16 (rows contiguous) -> (topk_idx [T, k] int32,
    topk_w [T, k] fp32)."""
    what = "moe_route_scores"
    shape, dev, k = x.shape, router.device, router.k
    if x.dtype is not torch.bfloat16 or len(shape) != 2 or shape[1] != router.H or x.get_device() != dev:
        raise QSMError(f"{what}: x must be [T, {router.H}] bf16 on the router's device")
    T = shape[0]
    ldx = shape[1] if x.is_contiguous() else _matrix(x, what)[3]
    on = _handle(dev, stream, what)
    if topk_idx is None:
        topk_idx = _empty(T, k, torch.int32, stream)
    elif (topk_idx.dtype is not torch.int32 or tuple(topk_idx.shape) != (T, k)
          or not topk_idx.is_contiguous() or topk_idx.get_device() != dev):
        raise QSMError(f"{what}: topk_idx must be a contiguous int32 [T, k] on x's device")
    if topk_w is None:
        topk_w = _empty(T, k, torch.float32, stream)
    elif (topk_w.dtype is not torch.float32 or tuple(topk_w.shape) != (T, k)
          or not topk_w.is_contiguous() or topk_w.get_device() != dev):
        raise QSMError(f"{what}: topk_w must be a contiguous fp32 [T, k] on x's device")
    if on not in router._ready.streams:
        router._ready.wait(on, stream)
    rc = (_lib or _load()).moe_route_scores(
        router.ref, x.data_ptr(), ldx, T, topk_idx.data_ptr(), topk_w.data_ptr(),
        _status(dev_status, dev, what), on)
    if rc:
        _check(rc, what)
    return topk_idx, topk_w


# ----------------------------------------------------------------- adapters

_LORA_DTYPES = {torch.bfloat16: 0, torch.float32: 2}


class LoraAdapters(_Fixed):
    """Low-rank adapters for one projection of K inputs and N outputs: a
    [n, rank, K] and b [n, N, rank] bf16, scale [n] fp32 or None (1), ranks [n]
    int32 or None: how many ranks of each adapter count (the others are not
    used, whatever they hold).  rank a multiple of 8, at most 128.  The contents
    may change (an adapter loaded into a place), the attributes not be replaced."""

    def __init__(self, a: torch.Tensor, b: torch.Tensor, scale=None, ranks=None):
        what = "LoraAdapters"
        if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
            raise QSMError(f"{what}: a must be [n, rank, K] and b [n, N, rank]")
        self.n, self.rank, self.K = a.shape
        self.N, self.device = b.shape[1], a.get_device()
        if (self.n < 1 or self.rank < 8 or self.rank % 8 or self.rank > 128 or self.K < 8 or self.K % 8
                or self.N < 1):
            raise QSMError(f"{what}: rank must be a multiple of 8 up to 128, K one of 8, n and N positive")
        for t in (a, b):
            if t.dtype is not torch.bfloat16 or not t.is_contiguous() or t.get_device() != self.device or self.device < 0:
                raise QSMError(f"{what}: a and b must be contiguous bf16 tensors on one GPU")
        _fp32(scale, (self.n,), self.device, f"{what}: scale")
        if ranks is not None and (ranks.dtype is not torch.int32 or tuple(ranks.shape) != (self.n,)
                                  or not ranks.is_contiguous() or ranks.get_device() != self.device):
            raise QSMError(f"{what}: ranks must be a contiguous int32 [n] on the adapters' device")
        self.a, self.b, self.scale, self.ranks = a, b, scale, ranks
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self.c = LoraC(self.n, self.rank, self.K, self.N, p(a), p(b), p(scale), p(ranks))
        self.ref = ctypes.byref(self.c)


def lora_add(x: torch.Tensor, adapters: LoraAdapters, ids: torch.Tensor, y=None, out=None,
             dtype=None, dev_status=None, stream=None) -> torch.Tensor:
    """out [T, N] = y [T, N] + scale * b (a x) of each token's adapter.
      x [T, K] bf16;  ids [T] int32, negative: no adapter
      y  the projection's output, bf16 or fp32, or None (zeros: then dtype, or out's
         type, or bf16);  out  None (a new tensor) or where to write: y itself is fine"""
    what = "lora_add"
    shape, dev, N = x.shape, adapters.device, adapters.N
    if x.dtype is not torch.bfloat16 or len(shape) != 2 or shape[1] != adapters.K or x.get_device() != dev:
        raise QSMError(f"{what}: x must be [T, {adapters.K}] bf16 on the adapters' device")
    T = shape[0]
    ldx = shape[1] if x.is_contiguous() else _matrix(x, what)[3]
    if ids.dtype is not torch.int32 or ids.shape != (T,) or not ids.is_contiguous() or ids.get_device() != dev:
        raise QSMError(f"{what}: ids must be a contiguous int32 [T] on x's device")
    on = _handle(dev, stream, what)
    kind = y.dtype if y is not None else out.dtype if out is not None else dtype or torch.bfloat16
    dt = _LORA_DTYPES.get(kind)
    if dt is None or (dtype is not None and dtype != kind):
        raise QSMError(f"{what}: y and out must be bf16 or fp32, and of dtype where it is given")
    yp, ldy = None, 0
    if y is not None:
        yp, ldy = y.data_ptr(), _ld(y, (T, N), dev, "lora_add: y")
    if out is None:
        out, ldo = _empty(T, N, kind, stream), N
    else:
        if out.dtype != kind:
            raise QSMError(f"{what}: out must be of y's type")
        ldo = _ld(out, (T, N), dev, "lora_add: out")
    rc = (_lib or _load()).lora_add(
        adapters.ref, x.data_ptr(), ldx, T, ids.data_ptr(), dt, yp, ldy, out.data_ptr(), ldo,
        _status(dev_status, dev, what), on)
    if rc:
        _check(rc, what)
    return out
