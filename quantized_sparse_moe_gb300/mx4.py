"""Binding of the MXFP4 calls of the qsmoe CUDA library: quantization,
4-bit products, few-row products with 16-bit activations, and the MoE layer
with MXFP4 weights (contracts in include/qsmoe.h).

As the rest of the binding, argument marshalling only: outputs and
workspaces are allocated with torch when the caller does not pass them, and a
non-zero status raises ``QSMError``.  What only shows on the device (a value
that is not finite) goes to dev_status, an int32 tensor; without one it is not
reported.  Import the names from the package."""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import QSMError, _check, lib, route_flags

BLOCK = 32            # columns per scale
TILE_ROWS = 128       # rows and columns of a scale tile
TILE_COLS = 128
TILE_BYTES = 512
GEMV_MAX_ROWS = 32
MOE_MAX_ROWS = 64     # of acts="bf16"

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_ACTS = {"bf16": 0, "mx4": 1}
_SEPARATE = 16        # with "bf16": never the one-launch form


def _acts(acts: str, one_launch: bool) -> int:
    return _ACTS.get(acts, -1) if one_launch or acts != "bf16" else _SEPARATE


class Mx4C(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("cols", ctypes.c_int32), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p)]


class Mx4LayerC(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("gate_up", Mx4C), ("down", Mx4C),
                ("shared_gate_up", Mx4C), ("shared_down", Mx4C),
                ("shared_gate", ctypes.c_void_p)]


def declare(L: ctypes.CDLL) -> None:
    """Argument and result types of the MXFP4 entry points of library L."""
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    M, st = ctypes.POINTER(Mx4C), ctypes.c_int
    L.mx4_scale_bytes.argtypes, L.mx4_scale_bytes.restype = [i32, i32], sz
    L.mx4_quantize.argtypes = [P, i32, i64, i32, i32, P, P, P, P]
    L.mx4_dequantize.argtypes = [M, i32, P, P]
    L.mx4_gemm.argtypes = [M, M, i32, P, i64, P, P]
    L.mx4_gemv.argtypes = [P, i64, i32, M, P, P, P]
    L.moe_mx4_workspace_bytes.argtypes = [ctypes.POINTER(Mx4LayerC), i32, i32]
    L.moe_mx4_workspace_bytes.restype = sz
    L.moe_mx4_forward.argtypes = [ctypes.POINTER(Mx4LayerC), P, i32, i32, P, P, i32,
                                  P, P, P, P, P, sz, P, P]
    L.moe_mx4_experts.argtypes = [ctypes.POINTER(Mx4LayerC), P, i32, i32, P, P, P, P, P, sz, P, P]
    for f in (L.mx4_quantize, L.mx4_dequantize, L.mx4_gemm, L.mx4_gemv, L.moe_mx4_forward,
              L.moe_mx4_experts):
        f.restype = st


# The calls below take a few microseconds of host time each, which is what
# bounds their smallest sizes: they look the library up once, read each
# property of a tensor once, pass plain integers, and allocate their outputs by
# the short way that torch has for strided CUDA tensors (a launch and an
# allocation take 5.2 us so, with torch.empty 8.5, with Tensor.new_empty more).
try:
    from torch._C._dynamo.guards import _empty_strided_cuda as _strided
except ImportError:  # a torch without it
    _strided = None
_lib = None
_stream_of = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_words: dict = {}


def _load():
    global _lib
    _lib = lib()
    return _lib


def _word(device: int) -> int:
    """A status word of the device, for the calls that are given none (it only
    ever collects bits)."""
    w = _words.get(device)
    if w is None:
        t = torch.zeros(1, dtype=torch.int32, device=f"cuda:{device}")
        w = _words[device] = (t.data_ptr(), t)
    return w[0]


def _empty(rows: int, cols: int, dtype, stream) -> torch.Tensor:
    """A [rows, cols] tensor on the current device, from the memory of the stream
    that will write it: what the current stream has given back may still be in
    use there, and another stream does not wait for that."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return torch.empty((rows, cols), dtype=dtype, device="cuda")
    if _strided is not None:
        return _strided((rows, cols), (cols or 1, 1), dtype)
    return torch.empty((rows, cols), dtype=dtype, device="cuda")


def _handle(dev: int, stream, what: str) -> int:
    """The stream to launch on: the given one, or the current one.  The library
    launches on the current device, so operands and stream have to be there."""
    if dev != _current_device():
        raise QSMError(f"{what}: the operands' device (cuda:{dev}) has to be the current one")
    if stream is None:
        return _stream_of(dev)
    if stream.device_index != dev:
        raise QSMError(f"{what}: the stream is not on the operands' device (cuda:{dev})")
    return stream.cuda_stream


def _status(t, dev: int, what: str) -> int:
    """The address of a status word to use: the caller's t, or the device's."""
    if t is None:
        return _word(dev)
    if t.dtype is not torch.int32 or t.get_device() != dev or t.numel() < 1:
        raise QSMError(f"{what}: dev_status must be an int32 tensor on the operands' device")
    return t.data_ptr()


def _fp32(t, shape, dev: int, what: str):
    """t, None or a contiguous fp32 tensor of that shape on the device."""
    if t is not None and (t.dtype is not torch.float32 or tuple(t.shape) != shape
                          or not t.is_contiguous() or t.get_device() != dev):
        raise QSMError(f"{what} must be contiguous fp32 {list(shape)} on the weights' device")
    return t


def _matrix(x: torch.Tensor, what: str):
    """(device, rows, columns, row stride) of a CUDA matrix whose rows are
    contiguous."""
    shape, stride, dev = x.shape, x.stride(), x.get_device()
    if len(shape) != 2 or dev < 0 or (stride[1] != 1 and shape[1] > 1):
        raise QSMError(f"{what}: needs a CUDA matrix with contiguous rows")
    rows, cols = shape
    return dev, rows, cols, stride[0] if rows > 1 else (cols + 7) // 8 * 8


def mx4_scale_bytes(rows: int, cols: int) -> int:
    """Bytes of the scale tiles of one [rows, cols] matrix."""
    return -(-rows // TILE_ROWS) * -(-cols // TILE_COLS) * TILE_BYTES


def mx4_tile_scales(scales: torch.Tensor) -> torch.Tensor:
    """Scale bytes [experts, rows, cols / 32] (or [rows, cols / 32]) in plain
    row order -> the tiles the library takes, rows and blocks padded with 0:
    once per weight, when a checkpoint is loaded."""
    s = scales if scales.dim() == 3 else scales[None]
    s = torch.nn.functional.pad(s, (0, -s.shape[2] % 4, 0, -s.shape[1] % TILE_ROWS))
    t = s.reshape(s.shape[0], -1, 4, 32, s.shape[2] // 4, 4)
    return t.permute(0, 1, 4, 3, 2, 5).reshape(-1).contiguous()


class _Fixed:
    """Attributes that cannot be replaced once they are set (`a.x -= 1`, which
    puts the same object back, is fine), but for those in _free."""
    _free: tuple = ()

    def __setattr__(self, name, value):
        if name in self.__dict__ and name not in self._free and self.__dict__[name] is not value:
            raise AttributeError(f"{type(self).__name__}: {name} cannot be replaced; make another one")
        super().__setattr__(name, value)


@dataclasses.dataclass(eq=False)
class Mx4Tensor(_Fixed):
    """An MXFP4 matrix, or `experts` of them: codes uint8
    [experts * rows, cols / 2] (any shape of that size) and scale tiles uint8,
    both contiguous on one GPU.  The calls use the addresses taken here: the
    contents may change, the attributes not be replaced."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int
    experts: int = 1

    def __post_init__(self):
        if self.cols % BLOCK or self.cols < BLOCK or self.rows < 0 or self.experts < 1:
            raise QSMError("Mx4Tensor: cols must be a positive multiple of 32")
        n = self.experts * self.rows * self.cols // 2
        sb = self.experts * mx4_scale_bytes(self.rows, self.cols)
        for t, size, what in ((self.codes, n, "codes"), (self.scales, sb, "scales")):
            if t.dtype != torch.uint8 or not t.is_contiguous() or t.numel() != size:
                raise QSMError(f"Mx4Tensor: {what} must be {size} contiguous bytes")
        self.device = self.codes.get_device()
        if self.device < 0 or self.scales.get_device() != self.device:
            raise QSMError("Mx4Tensor: codes and scales must be on one GPU")
        self.c = Mx4C(self.experts, self.rows, self.cols, self.codes.data_ptr(),
                      self.scales.data_ptr())
        self.ref = ctypes.byref(self.c)

    @classmethod
    def empty(cls, rows: int, cols: int, experts: int = 1, device="cuda") -> "Mx4Tensor":
        return cls(torch.empty((experts * rows, cols // 2), dtype=torch.uint8, device=device),
                   torch.empty(experts * mx4_scale_bytes(rows, cols), dtype=torch.uint8,
                               device=device), rows, cols, experts)

    @classmethod
    def _made(cls, codes, scales, rows: int, cols: int, device: int) -> "Mx4Tensor":
        """One matrix of buffers that need no checks (3 us less of a small call)."""
        t = cls.__new__(cls)
        c = Mx4C(1, rows, cols, codes.data_ptr(), scales.data_ptr())
        t.__dict__.update(codes=codes, scales=scales, rows=rows, cols=cols, experts=1, device=device,
                          c=c, ref=ctypes.byref(c))
        return t

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def _empty_mx4(rows: int, cols: int, device: int, stream) -> Mx4Tensor:
    """An Mx4Tensor on the current device, which `device` is (see _empty)."""
    if cols % BLOCK or cols < BLOCK:
        raise QSMError("Mx4Tensor: cols must be a positive multiple of 32")
    tiles = -(-rows // TILE_ROWS) * -(-cols // TILE_COLS)
    return Mx4Tensor._made(_empty(rows, cols // 2, torch.uint8, stream),
                           _empty(tiles, TILE_BYTES, torch.uint8, stream).view(-1), rows, cols, device)


def mx4_quantize(x: torch.Tensor, out: Mx4Tensor | None = None, dev_status=None,
                 stream=None) -> Mx4Tensor:
    """x [rows, cols] (bf16, fp16 or fp32) -> MXFP4."""
    dtype = _DTYPES.get(x.dtype)
    if dtype is None:
        raise QSMError("mx4_quantize: x must be bf16, fp16 or fp32")
    dev, rows, cols, ld = _matrix(x, "mx4_quantize")
    on = _handle(dev, stream, "mx4_quantize")
    if out is None:
        out = _empty_mx4(rows, cols, dev, stream)
    elif out.rows != rows or out.cols != cols or out.experts != 1 or out.device != dev:
        raise QSMError("mx4_quantize: out has another shape or device")
    rc = (_lib or _load()).mx4_quantize(
        x.data_ptr(), dtype, ld, rows, cols, out.c.codes, out.c.scales,
        _status(dev_status, dev, "mx4_quantize"), on)
    if rc:
        _check(rc, "mx4_quantize")
    return out


def mx4_dequantize(a: Mx4Tensor, dtype=torch.bfloat16, y=None, stream=None) -> torch.Tensor:
    """The values [experts * rows, cols] that a stands for."""
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise QSMError("mx4_dequantize: dtype must be bf16, fp16 or fp32")
    on = _handle(a.device, stream, "mx4_dequantize")
    if y is None:
        y = _empty(a.experts * a.rows, a.cols, dtype, stream)
    elif (y.dtype != dtype or not y.is_contiguous() or y.numel() != a.experts * a.rows * a.cols
          or y.get_device() != a.device):
        raise QSMError("mx4_dequantize: y must be contiguous, of a's size and device, and dtype")
    rc = (_lib or _load()).mx4_dequantize(a.ref, dt, y.data_ptr(), on)
    if rc:
        _check(rc, "mx4_dequantize")
    return y


def mx4_gemm(a: Mx4Tensor, w: Mx4Tensor, dtype=torch.bfloat16, y=None, dev_status=None,
             stream=None) -> torch.Tensor:
    """y [M, N] (bf16 or fp32) = a [M, K] w [N, K]^T."""
    M, N, dev = a.rows, w.rows, a.device
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise QSMError("mx4_gemm: dtype must be bf16 or fp32")
    if w.device != dev:
        raise QSMError("mx4_gemm: a and w are on different devices")
    on = _handle(dev, stream, "mx4_gemm")
    if y is None:
        y = _empty(M, N, dtype, stream)
        ld = N
    else:
        ydev, rows, cols, ld = _matrix(y, "mx4_gemm: y")
        if y.dtype != dtype or rows != M or cols != N or ydev != dev:
            raise QSMError("mx4_gemm: y must be [M, N] of dtype on the operands' device")
    rc = (_lib or _load()).mx4_gemm(
        a.ref, w.ref, _DTYPES[dtype], y.data_ptr(), ld,
        _status(dev_status, dev, "mx4_gemm"), on)
    if rc:
        _check(rc, "mx4_gemm")
    return y


def mx4_gemv(x: torch.Tensor, w: Mx4Tensor, y=None, dev_status=None, stream=None) -> torch.Tensor:
    """y [T, N] bf16 = x [T, K] w [N, K]^T for at most 32 rows of bf16 x."""
    if x.dtype is not torch.bfloat16:
        raise QSMError("mx4_gemv: x must be bf16")
    dev, T, K, ld = _matrix(x, "mx4_gemv")
    if K != w.cols or w.device != dev:
        raise QSMError("mx4_gemv: x and w differ in K or device")
    on = _handle(dev, stream, "mx4_gemv")
    if y is None:
        y = _empty(T, w.rows, torch.bfloat16, stream)
    elif (y.dtype != torch.bfloat16 or tuple(y.shape) != (T, w.rows) or not y.is_contiguous()
          or y.get_device() != dev):
        raise QSMError("mx4_gemv: y must be a contiguous bf16 [T, N] on x's device")
    rc = (_lib or _load()).mx4_gemv(
        x.data_ptr(), ld, T, w.ref, y.data_ptr(),
        _status(dev_status, dev, "mx4_gemv"), on)
    if rc:
        _check(rc, "mx4_gemv")
    return y


class Mx4Layer(_Fixed):
    """One MoE layer with MXFP4 weights (gate_up [E, 2I, H], down [E, H, I] and
    the shared expert's); keeps the tensors alive.  The weights' contents may
    change, the attributes not be replaced, but for the router's (w_router and
    logit_bias), which an Mx4Forward takes as they are when it is made."""
    _free = ("w_router", "logit_bias")

    def __init__(self, H, I, E, k, gate_up: Mx4Tensor, down: Mx4Tensor,
                 shared_gate_up: Mx4Tensor, shared_down: Mx4Tensor, w_router,
                 logit_bias=None, shared_gate=None):
        self.H, self.I, self.E, self.k = H, I, E, k
        self.w_router, self.logit_bias, self.shared_gate = w_router, logit_bias, shared_gate
        self.gate_up, self.down = gate_up, down
        self.shared_gate_up, self.shared_down = shared_gate_up, shared_down
        self.device = gate_up.device
        if any(m.device != self.device for m in (down, shared_gate_up, shared_down)):
            raise QSMError("Mx4Layer: the weights must be on one GPU")
        # what self.c points to
        self._keep = (gate_up, down, shared_gate_up, shared_down,
                      _fp32(shared_gate, (H,), self.device, "Mx4Layer: shared_gate"))
        self.c = Mx4LayerC(H, I, E, k, gate_up.c, down.c, shared_gate_up.c, shared_down.c,
                           None if shared_gate is None else shared_gate.data_ptr())

    @classmethod
    def quantize(cls, H, I, E, k, gate_up, down, shared_gate_up, shared_down, w_router,
                 logit_bias=None, shared_gate=None) -> "Mx4Layer":
        """From dense weights [E, 2I, H], [E, H, I], [1, 2I, H] and [1, H, I]."""
        def one(w):
            w = w.contiguous()  # row tiles of the experts follow one another: rows % 128 == 0
            t = mx4_quantize(w.reshape(-1, w.shape[2]))
            return Mx4Tensor(t.codes, t.scales, w.shape[1], w.shape[2], w.shape[0])
        if H % TILE_ROWS or I % TILE_ROWS:
            raise QSMError("Mx4Layer: H and I must be multiples of 128")
        return cls(H, I, E, k, one(gate_up), one(down), one(shared_gate_up), one(shared_down),
                   w_router, logit_bias, shared_gate)


def moe_mx4_workspace_bytes(layer: Mx4Layer, T: int, acts: str = "bf16", one_launch=True) -> int:
    """0 when the layer, T or acts is not supported (on the current device, which
    has to be the weights')."""
    _handle(layer.device, None, "moe_mx4_workspace_bytes")
    return int(lib().moe_mx4_workspace_bytes(ctypes.byref(layer.c), T, _acts(acts, one_launch)))


class Mx4Forward:
    """Buffers of one call of an MXFP4 MoE layer for T tokens, and the call.
    acts="bf16" (T <= 64) multiplies the weights with x and h unrounded,
    acts="mx4" with their MXFP4 forms.  One or two tokens with acts="bf16" run
    in one launch whose CTAs wait for one another, unless one_launch=False (for a
    GPU that runs other work beside the call).  With router, an MoERouter of the
    layer's H, E and k, the tokens are routed by its scores (always separate
    launches); the layer's own router, renormalize and bias_select_only are not
    used then.  Results: y (returned), topk_idx, topk_w, and y_f32 with want_f32."""

    def __init__(self, layer: Mx4Layer, T: int, acts: str = "bf16", device="cuda",
                 renormalize=True, want_f32=False, *, bias_select_only=False, one_launch=True,
                 router=None):
        if acts not in _ACTS:
            raise QSMError('Mx4Forward: acts must be "bf16" or "mx4"')
        if router is not None:
            if (router.H, router.E, router.k, router.device) != (layer.H, layer.E, layer.k, layer.device):
                raise QSMError("Mx4Forward: the router's H, E, k and device must be the layer's")
            one_launch = False
        self.router = router
        need = moe_mx4_workspace_bytes(layer, T, acts, one_launch)
        if T < 0 or (need == 0 and T > 0):
            raise QSMError("Mx4Forward: unsupported layer or token count")
        # the layer's own router as it is now (what the calls point to)
        self._router = (None, None) if router is not None else (
            _fp32(layer.w_router, (layer.E, layer.H), layer.device, "Mx4Forward: w_router"),
            _fp32(layer.logit_bias, (layer.E,), layer.device, "Mx4Forward: logit_bias"))
        if self._router[0] is None and router is None:
            raise QSMError("Mx4Forward: the layer has no router")
        self.layer, self.T, self.acts = layer, T, acts
        k, H = layer.k, layer.H
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, device=device)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=device)
        self.y = torch.empty((T, H), dtype=torch.bfloat16, device=device)
        self.y_f32 = torch.empty((T, H), dtype=torch.float32, device=device) if want_f32 else None
        self.workspace = torch.zeros(max(need, 256), dtype=torch.uint8, device=device)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=device)
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        if router is None:
            self._fn = lib().moe_mx4_forward
            self._mid = (T, _acts(acts, one_launch), p(layer.w_router), p(layer.logit_bias),
                         route_flags(renormalize, bias_select_only), p(self.topk_idx), p(self.topk_w))
        else:
            self._fn = lib().moe_mx4_experts
            self._mid = (T, _acts(acts, one_launch), p(self.topk_idx), p(self.topk_w))
        self._tail = (p(self.y_f32), p(self.workspace), self.workspace.numel(), p(self.dev_status))
        self._layer_ref = ctypes.byref(layer.c)
        self._device, self._shape = self.y.get_device(), self.y.shape
        if self._device != layer.device:
            raise QSMError("Mx4Forward: device is not the weights'")
        # the streams that are behind the zeroing of the buffers: this one, and
        # those that have waited for the event
        self._ready = {_stream_of(self._device)}
        self._zeroed = None
        if not torch.cuda.is_current_stream_capturing():
            self._zeroed = torch.cuda.Event()
            self._zeroed.record()

    def __call__(self, x: torch.Tensor, stream=None, out=None) -> torch.Tensor:
        """Run the layer on x [T, H] bf16; the result goes to out (a [T, H] bf16
        tensor, contiguous; x itself is fine) when given, else to self.y.  Returns it."""
        y = self.y if out is None else out
        for t in (x,) if out is None else (x, out):
            if (t.dtype is not torch.bfloat16 or t.shape != self._shape or not t.is_contiguous()
                    or t.get_device() != self._device):
                raise QSMError("Mx4Forward: x and out must be contiguous [T, H] bf16 tensors on "
                               "the layer's device")
        on = _handle(self._device, stream, "Mx4Forward")
        if on not in self._ready:
            self._wait_ready(on, stream)
        if self.router is not None:
            self.router.route(x, self.topk_idx, self.topk_w, self.dev_status, stream)
        rc = self._fn(self._layer_ref, x.data_ptr(), *self._mid, y.data_ptr(), *self._tail, on)
        if rc:
            _check(rc, "moe_mx4_forward" if self.router is None else "moe_mx4_experts")
        return y

    def _wait_ready(self, on: int, stream) -> None:
        """The first call on a stream waits for the zeroing.  A stream that is
        being captured cannot wait for what came before the capture: there the
        caller does it, with a call or a wait before the capture."""
        if self._zeroed is not None and not torch.cuda.is_current_stream_capturing():
            (torch.cuda.current_stream() if stream is None else stream).wait_event(self._zeroed)
            self._ready.add(on)
