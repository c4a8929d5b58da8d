"""Binding of the calls around the expert and projection products: the
residual stream with its norms (contracts in include/qsmoe.h).

As the rest of the binding, argument marshalling only: outputs are allocated
with torch when the caller does not pass them, and a non-zero status raises
``QSMError``.  What only shows on the device (a value that is not finite) goes
to dev_status, an int32 tensor; without one it is not reported.  Import the
names from the package."""
from __future__ import annotations

import ctypes

import torch

from . import QSMError, _check, lib
from .mx4 import (Mx4Tensor, _DTYPES, _empty, _Fixed, _fp32, _handle, _matrix,
                  _status)

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


def declare(L: ctypes.CDLL) -> None:
    """Argument and result types of the entry points of library L."""
    P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    L.residual_norm.argtypes = [ctypes.POINTER(ResidualNormC), i32, P, i64, P, i64, P, i64,
                                P, i64, P, i64, P, P, P]
    L.residual_norm.restype = ctypes.c_int


_lib = None


def _load():
    global _lib
    _lib = lib()
    return _lib


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
        dev, T, H, ldx = _matrix(x, what)
        xt = _DTYPES.get(x.dtype)
        if xt is None or H != self.H or dev != self.device:
            raise QSMError(f"{what}: x must be [T, {self.H}] bf16, fp16 or fp32 on cuda:{self.device}")
        on = _handle(dev, stream, what)
        yp = gp = op = hp = sp = None
        yt = gt = gate_kind = ldy = ldg = ldo = ldh = 0
        if y is not None:
            ydev, rows, cols, ldy = _matrix(y, what + ": y")
            yt = _DTYPES.get(y.dtype)
            if yt is None or rows != T or cols != H or ydev != dev:
                raise QSMError(f"{what}: y must be [T, H] bf16, fp16 or fp32 on x's device")
            yp = y.data_ptr()
        if gate is not None:
            gt = _DTYPES.get(gate.dtype)
            shape = gate.shape
            if y is None or gt is None or gate.get_device() != dev:
                raise QSMError(f"{what}: a gate needs a y, and must be bf16, fp16 or fp32 on x's device")
            if len(shape) == 1 and shape[0] == H and gate.is_contiguous():
                gate_kind, ldg = 1, 0
            elif len(shape) == 2 and shape[0] == T and shape[1] == 1 != H:
                gate_kind, ldg = 2, gate.stride(0)
            elif len(shape) == 2 and shape[0] == T and shape[1] == H:
                gate_kind, ldg = 1, _matrix(gate, what + ": gate")[3]
            else:
                raise QSMError(f"{what}: gate must be [H], [T, 1] or [T, H]")
            gp = gate.data_ptr()
        if x_out is None:
            if y is not None:
                x_out = _empty(T, H, x.dtype, stream)
                op, ldo = x_out.data_ptr(), H
        else:
            odev, rows, cols, ldo = _matrix(x_out, what + ": x_out")
            if x_out.dtype != x.dtype or rows != T or cols != H or odev != dev:
                raise QSMError(f"{what}: x_out must be [T, H] of x's type and device")
            op = x_out.data_ptr()
        ht = 0
        if self.pre is None:
            if h is not None:
                raise QSMError(f"{what}: without a pre there is no h")
        elif isinstance(h, torch.Tensor):
            hdev, rows, cols, ldh = _matrix(h, what + ": h")
            ht = _DTYPES.get(h.dtype)
            if ht is None or rows != T or cols != H or hdev != dev:
                raise QSMError(f"{what}: h must be [T, H] bf16, fp16 or fp32 on x's device")
            hp = h.data_ptr()
        elif isinstance(h, Mx4Tensor) or h == "mx4":
            ht = _MX4
            if h == "mx4":
                if stream is None:
                    h = Mx4Tensor.empty(T, H, device=x.device)
                else:  # as _empty
                    with torch.cuda.stream(stream):
                        h = Mx4Tensor.empty(T, H, device=x.device)
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
