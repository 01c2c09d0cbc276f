"""ctypes binding of the microscaled 4-bit (MXFP4) operators of libaqlm_mi355x.so.

Argument marshalling only, as in `_lib`: tensors are checked, and their
pointers and the current HIP stream go to the C entry points of
include/aqlm_mx.h, which states the format and every rule. There is no
fallback: a missing library or a failing call raises.

    codes, scales = mx_quantize(W)              # dense [out, in] -> MXFP4
    layer = MxLayer(codes, scales)              # or MxLayer.quantize(W)
    y = layer.forward(x)                        # x: [batch, in] float16 or bfloat16
    y = layer.forward_mx(x)                     # activations microscaled too
    dx = layer.grad_input(dy)                   # gradient through the frozen weights

Under autograd an x that requires a gradient gets it: forward, forward_mx, gemm,
gemv and mx_gemv_batched are recorded with grad_input as their backward
(forward_mx: straight through the quantisation). The weights are constants.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from ._lib import _check, load_library

MX_BLOCK = 32
MX_MAX_DIM = 1 << 21
MX_TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
MX_RULES = {"floor": 0, "ceil": 1}
MX_SYMBOLS = ("aqlm_mx_quantize", "aqlm_mx_dequant", "aqlm_mx_gemv_batched",
              "aqlm_mx_gemm_workspace_size", "aqlm_mx_gemm", "aqlm_mx_gemm_mx_workspace_size",
              "aqlm_mx_gemm_mx", "aqlm_mx_gemm_quant_workspace_size", "aqlm_mx_gemm_quant",
              "aqlm_mx_grad_input_workspace_size", "aqlm_mx_grad_input")

_HALVES = (torch.float16, torch.bfloat16)
_BYTES = (torch.uint8,)


class MxMatrixStruct(ctypes.Structure):
    """Mirror of struct aqlm_mx_matrix in include/aqlm_mx.h."""
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_ready: Optional[ctypes.CDLL] = None


def _lib() -> ctypes.CDLL:
    global _ready
    if _ready is None:
        lib = load_library()
        P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        M = ctypes.POINTER(MxMatrixStruct)
        lib.aqlm_mx_quantize.argtypes = [P, I32, I64, I64, I32, P, P, P]
        lib.aqlm_mx_dequant.argtypes = [M, I32, P, P]
        lib.aqlm_mx_gemv_batched.argtypes = [P, P, P, I32, I64, I32, P]
        for name in ("gemm", "gemm_mx", "gemm_quant", "grad_input"):
            getattr(lib, f"aqlm_mx_{name}_workspace_size").argtypes = [M, I64, ctypes.POINTER(I64)]
        lib.aqlm_mx_gemm.argtypes = [M, P, I64, P, I32, P, I64, P]
        lib.aqlm_mx_grad_input.argtypes = [M, P, I64, P, I32, P, I64, P]
        lib.aqlm_mx_gemm_mx.argtypes = [M, M, P, I32, P, I64, P]
        lib.aqlm_mx_gemm_quant.argtypes = [M, P, I64, I32, P, I32, P, I64, P]
        for name in MX_SYMBOLS:
            getattr(lib, name).restype = ctypes.c_int
        _ready = lib
    return _ready


# torch's own quick forms of torch.cuda.current_device and current_stream, where
# the installed torch has them
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(device: torch.device, fn, *args) -> None:
    """fn(*args, stream) on the device's current stream, with the device current."""
    index, before = device.index, _current_device()
    if before == index:
        status = fn(*args, _current_stream(index))
    else:
        torch.cuda.set_device(index)
        try:
            status = fn(*args, _current_stream(index))
        finally:
            torch.cuda.set_device(before)
    if status:
        _check(status)


def _check_dense(t: torch.Tensor, what: str, dtypes, shape=None) -> None:
    if t.dtype not in dtypes or t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        names = ", ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{what} must be a contiguous 2-D tensor on the GPU, of type {names}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}, not {list(t.shape)}")


def _check_packed(codes: torch.Tensor, scales: torch.Tensor) -> Tuple[int, int]:
    _check_dense(codes, "codes", _BYTES)
    _check_dense(scales, "scales", _BYTES)
    rows, half = codes.shape
    if half < MX_BLOCK // 2 or half % (MX_BLOCK // 2) or scales.shape != (rows, half // (MX_BLOCK // 2)):
        raise ValueError("codes are [rows, cols/2] and scales [rows, cols/32], cols a multiple of 32")
    if codes.device != scales.device:
        raise ValueError("codes and scales must be on one device")
    return rows, 2 * half


def _output(out: Optional[torch.Tensor], shape, dtype, device) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _check_dense(out, "out", (dtype,), shape)
    if out.device != device:
        raise ValueError("out must be on the inputs' device")
    return out


def mx_quantize(x: torch.Tensor, rule: str = "floor",
                out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None
                ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes [rows, cols/2], scales [rows, cols/32]), both uint8, of a dense matrix.

    x is float16, bfloat16 or float32, cols a multiple of 32. rule "floor" is
    the format's own scale (values above 6 scales are held as 6), "ceil" the
    smallest scale that clips nothing."""
    _check_dense(x, "x", tuple(MX_TYPES))
    rows, cols = x.shape
    if rule not in MX_RULES:
        raise ValueError(f"rule must be one of {sorted(MX_RULES)}")
    if cols < MX_BLOCK or cols % MX_BLOCK:
        raise ValueError("cols must be a multiple of 32")
    codes = _output(None if out is None else out[0], (rows, cols // 2), torch.uint8, x.device)
    scales = _output(None if out is None else out[1], (rows, cols // MX_BLOCK), torch.uint8, x.device)
    _call(x.device, _lib().aqlm_mx_quantize, x.data_ptr(), MX_TYPES[x.dtype], rows, cols,
          MX_RULES[rule], codes.data_ptr(), scales.data_ptr())
    return codes, scales


def mx_dequant(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.float16,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The dense [rows, cols] matrix of a microscaled one, in float16, bfloat16 or float32."""
    rows, cols = _check_packed(codes, scales)
    if dtype not in MX_TYPES:
        raise ValueError("dtype must be float16, bfloat16 or float32")
    W = _output(out, (rows, cols), dtype, codes.device)
    m = MxMatrixStruct(rows, cols, codes.data_ptr(), scales.data_ptr())
    _call(codes.device, _lib().aqlm_mx_dequant, ctypes.byref(m), MX_TYPES[dtype], W.data_ptr())
    return W


class _Recorded(torch.autograd.Function):
    """Products of layers with one x each, and for backward each layer's grad_input."""

    @staticmethod
    def forward(ctx, products, layers, *xs):
        ctx.layers = layers
        ctx.set_materialize_grads(False)
        return tuple(products(xs))

    @staticmethod
    @once_differentiable
    def backward(ctx, *dys):
        grads = []
        for layer, dy, wanted in zip(ctx.layers, dys, ctx.needs_input_grad[2:]):
            if dy is None or not wanted:
                grads.append(None)
                continue
            dy = dy.contiguous()
            if dy.data_ptr() % 16:  # a part of a larger gradient
                dy = dy.clone()
            grads.append(layer.grad_input(dy))
        return (None, None, *grads)


def _record(products, layers, xs, outs):
    """products(xs), called again inside of the recording, as results of autograd's."""
    if outs is not None:
        raise ValueError("out takes no part in autograd: x must not require a gradient")
    return _Recorded.apply(products, layers, *xs)


class MxLayer:
    """A linear layer [out, in] whose weights are a microscaled matrix.

    codes [out, in/2] and scales [out, in/32], both uint8, as mx_quantize gives
    them. Activations are float16 or bfloat16 and results have their type."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        rows, cols = _check_packed(codes, scales)
        if rows < 1 or rows > MX_MAX_DIM or cols > MX_MAX_DIM:
            raise ValueError(f"a layer has 1 to {MX_MAX_DIM} rows and at most as many columns")
        self.codes, self.scales = codes, scales
        self.out_features, self.in_features = int(rows), int(cols)
        self.device = codes.device
        self._struct = MxMatrixStruct(rows, cols, codes.data_ptr(), scales.data_ptr())
        self._ref = ctypes.byref(self._struct)
        self._raw = bytes(self._struct)
        self._ws_bytes = {}  # (operator, batch) -> bytes: a rule of sizes alone

    @classmethod
    def quantize(cls, W: torch.Tensor, rule: str = "floor") -> "MxLayer":
        """The layer of a dense weight matrix [out, in]."""
        return cls(*mx_quantize(W, rule))

    def dequant(self, dtype: torch.dtype = torch.float16,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
        return mx_dequant(self.codes, self.scales, dtype, out)

    def _check_half(self, t: torch.Tensor, what: str, cols: int) -> None:
        _check_dense(t, what, _HALVES)
        if t.shape[1] != cols:
            raise ValueError(f"{what} must be [batch, {cols}]")
        if t.device != self.device:
            raise ValueError(f"{what} must be on the layer's device")

    def workspace_bytes(self, batch: int, op: str = "gemm") -> int:
        """Device workspace of gemm, gemm_mx, gemm_quant or grad_input at this batch (0: none)."""
        need = self._ws_bytes.get((op, batch))
        if need is None:
            n = ctypes.c_int64(0)
            _check(getattr(_lib(), f"aqlm_mx_{op}_workspace_size")(self._ref, batch, ctypes.byref(n)))
            need = n.value
            if len(self._ws_bytes) >= 1024:
                self._ws_bytes.clear()
            self._ws_bytes[(op, batch)] = need
        return need

    def _workspace(self, batch: int, op: str) -> Tuple[Optional[torch.Tensor], Optional[int], int]:
        need = self.workspace_bytes(batch, op)
        if not need:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        return ws, ws.data_ptr(), need

    def gemv(self, x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y = x . W^T for 1..8 activation rows."""
        return mx_gemv_batched([self], [x], None if out is None else [out])[0]

    def gemm(self, x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y = x . W^T for any number of activation rows; a workspace, where the
        call needs one, comes from torch's allocator on the current stream."""
        self._check_half(x, "x", self.in_features)
        if x.requires_grad and torch.is_grad_enabled():
            return _record(lambda xs: [self.gemm(xs[0])], (self,), (x,), out)[0]
        batch = x.shape[0]
        y = _output(out, (batch, self.out_features), x.dtype, self.device)
        ws, ptr, need = self._workspace(batch, "gemm")
        _call(self.device, _lib().aqlm_mx_gemm, self._ref, x.data_ptr(), batch, y.data_ptr(),
              MX_TYPES[x.dtype], ptr, need)
        return y

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """y = x . W^T, x [batch, in] float16 or bfloat16."""
        return self.gemm(x)

    def gemm_mx(self, codes: torch.Tensor, scales: torch.Tensor,
                dtype: torch.dtype = torch.float16,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y = x . W^T with microscaled activations (codes, scales), y of `dtype`."""
        batch, cols = _check_packed(codes, scales)
        if cols != self.in_features or codes.device != self.device:
            raise ValueError(f"the activations must have {self.in_features} columns, on the layer's "
                             "device")
        if dtype not in _HALVES:
            raise ValueError("dtype must be float16 or bfloat16")
        y = _output(out, (batch, self.out_features), dtype, self.device)
        xs = MxMatrixStruct(batch, cols, codes.data_ptr(), scales.data_ptr())
        ws, ptr, need = self._workspace(batch, "gemm_mx")
        _call(self.device, _lib().aqlm_mx_gemm_mx, self._ref, ctypes.byref(xs), y.data_ptr(),
              MX_TYPES[dtype], ptr, need)
        return y

    def forward_mx(self, x: torch.Tensor, rule: str = "floor",
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y = Q(x) . W^T: the activations quantised by mx_quantize's rule, then the product of
        gemm_mx, in one call."""
        self._check_half(x, "x", self.in_features)
        if rule not in MX_RULES:
            raise ValueError(f"rule must be one of {sorted(MX_RULES)}")
        if x.requires_grad and torch.is_grad_enabled():
            return _record(lambda xs: [self.forward_mx(xs[0], rule)], (self,), (x,), out)[0]
        batch = x.shape[0]
        y = _output(out, (batch, self.out_features), x.dtype, self.device)
        ws, ptr, need = self._workspace(batch, "gemm_quant")
        _call(self.device, _lib().aqlm_mx_gemm_quant, self._ref, x.data_ptr(), batch,
              MX_RULES[rule], y.data_ptr(), MX_TYPES[x.dtype], ptr, need)
        return y

    def grad_input(self, dy: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """dx = dy . W: the gradient of forward(x) with respect to x, and the
        straight-through one of forward_mx(x). Not recorded by autograd itself."""
        self._check_half(dy, "dy", self.out_features)
        batch = dy.shape[0]
        dx = _output(out, (batch, self.in_features), dy.dtype, self.device)
        ws, ptr, need = self._workspace(batch, "grad_input")
        _call(self.device, _lib().aqlm_mx_grad_input, self._ref, dy.data_ptr(), batch, dx.data_ptr(),
              MX_TYPES[dy.dtype], ptr, need)
        return dx


def mx_gemv_batched(layers, xs, outs=None):
    """y_i = x_i . W_i^T for several microscaled layers in one call.

    layers: sequence of MxLayer; xs: one [batch, in_i] tensor per layer (batch 0
    to 8 and type shared, may repeat); outs: optional [batch, out_i] tensors.
    Returns the list of outputs; without outs, those of layers of one size are
    parts of one allocation."""
    n = len(layers)
    if len(xs) != n or (outs is not None and len(outs) != n):
        raise ValueError("one x (and one out) per layer")
    if n == 0:
        return []
    device = layers[0].device
    layers[0]._check_half(xs[0], "x", layers[0].in_features)
    batch, dtype = xs[0].shape[0], xs[0].dtype
    seen, seen_cols, record = xs[0], layers[0].in_features, xs[0].requires_grad
    for L, x in zip(layers, xs):
        if x is seen and L.in_features == seen_cols and L.device == device:
            continue  # the x of the layer before, as with query, key and value
        L._check_half(x, "x", L.in_features)
        if x.shape[0] != batch or x.dtype != dtype or L.device != device:
            raise ValueError("all layers share the batch size, the type and the device")
        seen, seen_cols, record = x, L.in_features, record or x.requires_grad
    if record and torch.is_grad_enabled():
        def products(given):  # (not parts of one allocation, which could not be changed in place)
            return mx_gemv_batched(layers, given, [
                torch.empty((batch, L.out_features), dtype=dtype, device=device) for L in layers])
        return list(_record(products, tuple(layers), xs, outs))
    sizes = [L.out_features for L in layers]
    if outs is not None:
        ys = [_output(o, (batch, k), dtype, device) for o, k in zip(outs, sizes)]
    elif n > 1 and min(sizes) == max(sizes) and batch * sizes[0] % 8 == 0:  # (16-byte parts)
        ys = list(torch.empty((n, batch, sizes[0]), dtype=dtype, device=device).unbind(0))
    else:
        ys = [torch.empty((batch, k), dtype=dtype, device=device) for k in sizes]
    _call(device, _lib().aqlm_mx_gemv_batched, b"".join([L._raw for L in layers]),
          struct.pack(f"{n}P", *[x.data_ptr() for x in xs]),
          struct.pack(f"{n}P", *[y.data_ptr() for y in ys]), n, batch, MX_TYPES[dtype])
    return ys
