"""Binding of the MXFP4 calls of the qsmoe CUDA library: quantization,
4-bit products, few-row products with 16-bit activations, and the MoE layer
with MXFP4 weights (contracts in include/qsmoe.h).

As the rest of the binding, argument marshalling only: outputs and
workspaces are allocated with torch when the caller does not pass them, and a
non-zero status raises ``QSMError``.  Import the names from the package."""
from __future__ import annotations

import ctypes
import dataclasses

import torch

BLOCK = 32            # columns per scale
TILE_ROWS = 128       # rows and columns of a scale tile
TILE_COLS = 128
TILE_BYTES = 512
GEMV_MAX_ROWS = 32
MOE_MAX_ROWS = 64     # of acts="bf16"

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_ACTS = {"bf16": 0, "mx4": 1}


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
    for f in (L.mx4_quantize, L.mx4_dequantize, L.mx4_gemm, L.mx4_gemv, L.moe_mx4_forward):
        f.restype = st


def _q():
    import quantized_sparse_moe_gb300 as q
    return q


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


@dataclasses.dataclass
class Mx4Tensor:
    """An MXFP4 matrix, or `experts` of them: codes uint8
    [experts * rows, cols / 2] (any shape of that size) and scale tiles uint8,
    both contiguous on one GPU."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int
    experts: int = 1

    def __post_init__(self):
        if self.cols % BLOCK or self.cols < BLOCK or self.rows < 0 or self.experts < 1:
            raise _q().QSMError("Mx4Tensor: cols must be a positive multiple of 32")
        n = self.experts * self.rows * self.cols // 2
        sb = self.experts * mx4_scale_bytes(self.rows, self.cols)
        for t, size, what in ((self.codes, n, "codes"), (self.scales, sb, "scales")):
            if t.dtype != torch.uint8 or not t.is_contiguous() or t.numel() != size:
                raise _q().QSMError(f"Mx4Tensor: {what} must be {size} contiguous bytes")
        self.c = Mx4C(self.experts, self.rows, self.cols, self.codes.data_ptr(),
                      self.scales.data_ptr())

    @classmethod
    def empty(cls, rows: int, cols: int, experts: int = 1, device="cuda") -> "Mx4Tensor":
        return cls(torch.empty((experts * rows, cols // 2), dtype=torch.uint8, device=device),
                   torch.empty(experts * mx4_scale_bytes(rows, cols), dtype=torch.uint8,
                               device=device), rows, cols, experts)

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


_status_words: dict = {}


def _word(dev_status, device):
    """The caller's status word, or one per device that the calls without
    one share (it only ever collects bits)."""
    if dev_status is not None:
        return dev_status.data_ptr()
    w = _status_words.get(device)
    if w is None:
        w = _status_words[device] = torch.zeros(1, dtype=torch.int32, device=device)
    return w.data_ptr()


def _rows(x: torch.Tensor, what: str):
    """(row stride) of a matrix whose rows are contiguous."""
    if x.dim() != 2 or x.stride(1) != 1 or not x.is_cuda:
        raise _q().QSMError(f"{what}: x must be a CUDA matrix with contiguous rows")
    return x.stride(0) if x.shape[0] > 1 else max(x.shape[1], 8)


def _raw_stream(stream, device):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


def mx4_quantize(x: torch.Tensor, out: Mx4Tensor | None = None, dev_status=None,
                 stream=None) -> Mx4Tensor:
    """x [rows, cols] (bf16, fp16 or fp32) -> MXFP4."""
    q = _q()
    if x.dtype not in _DTYPES:
        raise q.QSMError("mx4_quantize: x must be bf16, fp16 or fp32")
    ld = _rows(x, "mx4_quantize")
    rows, cols = x.shape
    if out is None:
        out = Mx4Tensor.empty(rows, cols, device=x.device)
    elif out.rows != rows or out.cols != cols or out.experts != 1:
        raise q.QSMError("mx4_quantize: out has another shape")
    q._check(q.lib().mx4_quantize(x.data_ptr(), _DTYPES[x.dtype], ld, rows, cols,
                                  out.c.codes, out.c.scales, _word(dev_status, x.device),
                                  _raw_stream(stream, x.device)), "mx4_quantize")
    return out


def mx4_dequantize(a: Mx4Tensor, dtype=torch.bfloat16, y=None, stream=None) -> torch.Tensor:
    """The values [experts * rows, cols] that a stands for."""
    q = _q()
    if dtype not in _DTYPES:
        raise q.QSMError("mx4_dequantize: dtype must be bf16, fp16 or fp32")
    if y is None:
        y = torch.empty((a.experts * a.rows, a.cols), dtype=dtype, device=a.codes.device)
    elif y.dtype != dtype or not y.is_contiguous() or y.numel() != a.experts * a.rows * a.cols:
        raise q.QSMError("mx4_dequantize: y must be contiguous, of a's size and dtype")
    q._check(q.lib().mx4_dequantize(ctypes.byref(a.c), _DTYPES[dtype], y.data_ptr(),
                                    _raw_stream(stream, y.device)), "mx4_dequantize")
    return y


def mx4_gemm(a: Mx4Tensor, w: Mx4Tensor, dtype=torch.bfloat16, y=None, dev_status=None,
             stream=None) -> torch.Tensor:
    """y [M, N] (bf16 or fp32) = a [M, K] w [N, K]^T."""
    q = _q()
    if y is None:
        y = torch.empty((a.rows, w.rows), dtype=dtype, device=a.codes.device)
    elif y.dtype != dtype or tuple(y.shape) != (a.rows, w.rows) or y.stride(1) != 1:
        raise q.QSMError("mx4_gemm: y must be [M, N] of dtype with contiguous rows")
    if dtype not in (torch.bfloat16, torch.float32):
        raise q.QSMError("mx4_gemm: dtype must be bf16 or fp32")
    ld = y.stride(0) if a.rows > 1 else max(w.rows, 1)
    q._check(q.lib().mx4_gemm(ctypes.byref(a.c), ctypes.byref(w.c), _DTYPES[dtype], y.data_ptr(),
                              ld, _word(dev_status, y.device), _raw_stream(stream, y.device)),
             "mx4_gemm")
    return y


def mx4_gemv(x: torch.Tensor, w: Mx4Tensor, y=None, dev_status=None, stream=None) -> torch.Tensor:
    """y [T, N] bf16 = x [T, K] w [N, K]^T for at most 32 rows of bf16 x."""
    q = _q()
    if x.dtype != torch.bfloat16:
        raise q.QSMError("mx4_gemv: x must be bf16")
    ld = _rows(x, "mx4_gemv")
    if x.shape[1] != w.cols:
        raise q.QSMError("mx4_gemv: x and w differ in K")
    if y is None:
        y = torch.empty((x.shape[0], w.rows), dtype=torch.bfloat16, device=x.device)
    elif y.dtype != torch.bfloat16 or tuple(y.shape) != (x.shape[0], w.rows) or not y.is_contiguous():
        raise q.QSMError("mx4_gemv: y must be a contiguous bf16 [T, N]")
    q._check(q.lib().mx4_gemv(x.data_ptr(), ld, x.shape[0], ctypes.byref(w.c), y.data_ptr(),
                              _word(dev_status, x.device), _raw_stream(stream, x.device)),
             "mx4_gemv")
    return y


class Mx4Layer:
    """One MoE layer with MXFP4 weights (gate_up [E, 2I, H], down [E, H, I] and
    the shared expert's); keeps the tensors alive."""

    def __init__(self, H, I, E, k, gate_up: Mx4Tensor, down: Mx4Tensor,
                 shared_gate_up: Mx4Tensor, shared_down: Mx4Tensor, w_router,
                 logit_bias=None, shared_gate=None):
        self.H, self.I, self.E, self.k = H, I, E, k
        self.w_router, self.logit_bias, self.shared_gate = w_router, logit_bias, shared_gate
        self.gate_up, self.down = gate_up, down
        self.shared_gate_up, self.shared_down = shared_gate_up, shared_down
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
            raise _q().QSMError("Mx4Layer: H and I must be multiples of 128")
        return cls(H, I, E, k, one(gate_up), one(down), one(shared_gate_up), one(shared_down),
                   w_router, logit_bias, shared_gate)


def moe_mx4_workspace_bytes(layer: Mx4Layer, T: int, acts: str = "bf16") -> int:
    """0 when the layer, T or acts is not supported."""
    return int(_q().lib().moe_mx4_workspace_bytes(ctypes.byref(layer.c), T, _ACTS[acts]))


class Mx4Forward:
    """Buffers of one call of an MXFP4 MoE layer for T tokens, and the call.
    acts="bf16" (T <= 64) multiplies the weights with x and h unrounded,
    acts="mx4" with their MXFP4 forms.  Results: y (returned), topk_idx,
    topk_w, and y_f32 with want_f32."""

    def __init__(self, layer: Mx4Layer, T: int, acts: str = "bf16", device="cuda",
                 renormalize=True, want_f32=False, *, bias_select_only=False):
        q = _q()
        if acts not in _ACTS:
            raise q.QSMError('Mx4Forward: acts must be "bf16" or "mx4"')
        need = moe_mx4_workspace_bytes(layer, T, acts)
        if need == 0 and T > 0:
            raise q.QSMError("Mx4Forward: unsupported layer or token count")
        self.layer, self.T, self.acts = layer, T, acts
        k, H = layer.k, layer.H
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, device=device)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=device)
        self.y = torch.empty((T, H), dtype=torch.bfloat16, device=device)
        self.y_f32 = torch.empty((T, H), dtype=torch.float32, device=device) if want_f32 else None
        self.workspace = torch.zeros(max(need, 256), dtype=torch.uint8, device=device)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=device)
        self._fn = q.lib().moe_mx4_forward
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self._mid = (T, _ACTS[acts], p(layer.w_router), p(layer.logit_bias),
                     q.route_flags(renormalize, bias_select_only), p(self.topk_idx), p(self.topk_w))
        self._tail = (p(self.y_f32), p(self.workspace), self.workspace.numel(), p(self.dev_status))
        self._layer_ref = ctypes.byref(layer.c)

    def __call__(self, x: torch.Tensor, stream=None, out=None) -> torch.Tensor:
        """Run the layer on x [T, H] bf16; the result goes to out (a [T, H] bf16
        tensor, contiguous) when given, else to self.y.  Returns it."""
        y = self.y if out is None else out
        if (x.dtype != torch.bfloat16 or not x.is_contiguous() or x.shape != self.y.shape
                or (out is not None and (out.dtype != torch.bfloat16 or not out.is_contiguous()
                                         or out.shape != self.y.shape))):
            raise _q().QSMError("Mx4Forward: x and out must be contiguous [T, H] bf16 tensors")
        rc = self._fn(self._layer_ref, x.data_ptr(), *self._mid, y.data_ptr(), *self._tail,
                      _raw_stream(stream, y.device))
        if rc:
            _q()._check(rc, "moe_mx4_forward")
        return y
