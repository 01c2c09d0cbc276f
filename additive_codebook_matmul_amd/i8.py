"""ctypes binding of the 8-bit integer (int8) operators of libaqlm_mi355x.so.

Argument marshalling only, as in `_lib`: tensors are checked, and their
pointers and the current HIP stream go to the C entry points of
include/aqlm_i8.h, which states the format and every rule. There is no
fallback: a missing library or a failing call raises.

    codes, scales = i8_quantize(W)              # dense [out, in] -> int8 rows
    layer = I8Layer(codes, scales)              # or I8Layer.quantize(W)
    y = layer.forward(x)                        # x: [batch, in] float16 or bfloat16
    dx = layer.grad_input(dy)                   # gradient through the frozen weights

    block = I8Gated(gate, up, "silu")           # two I8Layers of one size
    h = block.forward(x)                        # silu(gate(x)) * up(x), one pass
    y = down.forward(h)

Under autograd an x that requires a gradient gets it, straight through the
quantisation of the activations: I8Layer.forward and I8Gated.forward are recorded.
The weights are constants. What quantisation, expansion, gemm_i8, forward_saving and
grad_input return is outside autograd. Forward-mode derivatives are not computed: a
tensor that carries a tangent is refused. (As with torch's own
operations, a backward pass that is captured into a HIP graph must meet no eager
graph of the same leaves that is still alive: torch then accumulates into them on
the eager graph's stream.)
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from ._lib import _check, load_library
from .mx import _HALVES, _call, _check_dense, _output, _record, _refuse_tangent

I8_MAX_DIM = 1 << 21
I8_MAX_COLS = (1 << 17) - 16
I8_TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
I8_ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
I8_SYMBOLS = ("aqlm_i8_quantize", "aqlm_i8_dequant", "aqlm_i8_gemm_workspace_size", "aqlm_i8_gemm",
              "aqlm_i8_gemm_quant_workspace_size", "aqlm_i8_gemm_quant", "aqlm_i8_gated_workspace_size",
              "aqlm_i8_gated", "aqlm_i8_grad_input_workspace_size", "aqlm_i8_grad_input",
              "aqlm_i8_gated_grad_workspace_size", "aqlm_i8_gated_grad")

_INT8 = (torch.int8,)
_FLOAT = (torch.float32,)


class I8MatrixStruct(ctypes.Structure):
    """Mirror of struct aqlm_i8_matrix in include/aqlm_i8.h."""
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_ready: Optional[ctypes.CDLL] = None


def _lib() -> ctypes.CDLL:
    global _ready
    if _ready is None:
        lib = load_library()
        P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        M, N = ctypes.POINTER(I8MatrixStruct), ctypes.POINTER(ctypes.c_int64)
        lib.aqlm_i8_quantize.argtypes = [P, I32, I64, I64, P, P, P]
        lib.aqlm_i8_dequant.argtypes = [M, I32, P, P]
        for name in ("gemm", "gemm_quant", "grad_input"):
            getattr(lib, f"aqlm_i8_{name}_workspace_size").argtypes = [M, I64, N]
        for name in ("gated", "gated_grad"):
            getattr(lib, f"aqlm_i8_{name}_workspace_size").argtypes = [M, M, I64, N]
        lib.aqlm_i8_gemm.argtypes = [M, M, P, I32, P, I64, P]
        lib.aqlm_i8_gemm_quant.argtypes = [M, P, I64, P, I32, P, I64, P]
        lib.aqlm_i8_grad_input.argtypes = [M, P, I64, P, I32, P, I64, P]
        lib.aqlm_i8_gated.argtypes = [M, M, P, I64, I32, P, P, P, I32, P, I64, P]
        lib.aqlm_i8_gated_grad.argtypes = [M, M, P, P, P, I64, I32, P, I32, P, I64, P]
        for name in I8_SYMBOLS:
            getattr(lib, name).restype = ctypes.c_int
        _ready = lib
    return _ready


def _check_packed(codes: torch.Tensor, scales: torch.Tensor) -> Tuple[int, int]:
    _check_dense(codes, "codes", _INT8)
    rows, cols = codes.shape
    if (scales.dtype != torch.float32 or scales.shape != (rows,) or not scales.is_contiguous()
            or scales.device != codes.device):
        raise ValueError("scales must be float32 [rows], contiguous and on the codes' device")
    _refuse_tangent(scales, "scales")
    if cols < 16 or cols % 16:
        raise ValueError("cols must be a multiple of 16")
    return rows, cols


def _check_act(activation: str) -> int:
    if activation not in I8_ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(I8_ACTIVATIONS)}")
    return I8_ACTIVATIONS[activation]


def i8_quantize(x: torch.Tensor, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None
                ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes [rows, cols] int8, scales [rows] float32) of a dense matrix.

    x is float16, bfloat16 or float32, cols a multiple of 16. A row's largest
    magnitude becomes 127 or -127. Not recorded by autograd."""
    _check_dense(x, "x", tuple(I8_TYPES))
    rows, cols = x.shape
    if cols < 16 or cols % 16:
        raise ValueError("cols must be a multiple of 16")
    codes = _output(None if out is None else out[0], (rows, cols), torch.int8, x.device)
    if out is None:
        scales = torch.empty(rows, dtype=torch.float32, device=x.device)
    else:
        scales = out[1]
        _check_packed(codes, scales)
    _call(x.device, _lib().aqlm_i8_quantize, x.data_ptr(), I8_TYPES[x.dtype], rows, cols,
          codes.data_ptr(), scales.data_ptr())
    return codes, scales


def i8_dequant(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.float16,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The dense [rows, cols] matrix of an int8 one, in float16, bfloat16 or float32. Not recorded
    by autograd."""
    rows, cols = _check_packed(codes, scales)
    if dtype not in I8_TYPES:
        raise ValueError("dtype must be float16, bfloat16 or float32")
    W = _output(out, (rows, cols), dtype, codes.device)
    m = I8MatrixStruct(rows, cols, codes.data_ptr(), scales.data_ptr())
    _call(codes.device, _lib().aqlm_i8_dequant, ctypes.byref(m), I8_TYPES[dtype], W.data_ptr())
    return W


class _Workspaces:
    """Sizes and allocations of the workspaces of a layer's or block's calls."""

    def __init__(self, *refs):
        self._refs = refs
        self._ws_bytes = {}  # (operator, batch) -> bytes: a rule of sizes alone

    def workspace_bytes(self, batch: int, op: str) -> int:
        need = self._ws_bytes.get((op, batch))
        if need is None:
            n = ctypes.c_int64(0)
            _check(getattr(_lib(), f"aqlm_i8_{op}_workspace_size")(*self._refs, batch, ctypes.byref(n)))
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

    def _check_half(self, t: torch.Tensor, what: str, cols: int) -> None:
        _check_dense(t, what, _HALVES)
        if t.shape[1] != cols:
            raise ValueError(f"{what} must be [batch, {cols}]")
        if t.device != self.device:
            raise ValueError(f"{what} must be on the layer's device")


class I8Layer(_Workspaces):
    """A linear layer [out, in] whose weights are an int8 matrix.

    codes [out, in] int8 and scales [out] float32, as i8_quantize gives them.
    Activations are float16 or bfloat16 and results have their type. Layers of one
    input (query, key and value) may be joined along `out`: the scales are each
    channel's own."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        rows, cols = _check_packed(codes, scales)
        if rows < 1 or rows > I8_MAX_DIM or cols > I8_MAX_COLS:
            raise ValueError(f"a layer has 1 to {I8_MAX_DIM} rows and at most {I8_MAX_COLS} columns")
        self.codes, self.scales = codes, scales
        self.out_features, self.in_features = int(rows), int(cols)
        self.device = codes.device
        self._struct = I8MatrixStruct(rows, cols, codes.data_ptr(), scales.data_ptr())
        self._ref = ctypes.byref(self._struct)
        super().__init__(self._ref)

    @classmethod
    def quantize(cls, W: torch.Tensor) -> "I8Layer":
        """The layer of a dense weight matrix [out, in]."""
        return cls(*i8_quantize(W))

    def dequant(self, dtype: torch.dtype = torch.float16,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
        return i8_dequant(self.codes, self.scales, dtype, out)

    def gemm_i8(self, codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.float16,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y = x . W^T with int8 activations (codes, scales), y of `dtype`."""
        batch, cols = _check_packed(codes, scales)
        if cols != self.in_features or codes.device != self.device:
            raise ValueError(f"the activations must have {self.in_features} columns, on the layer's "
                             "device")
        if dtype not in _HALVES:
            raise ValueError("dtype must be float16 or bfloat16")
        y = _output(out, (batch, self.out_features), dtype, self.device)
        xs = I8MatrixStruct(batch, cols, codes.data_ptr(), scales.data_ptr())
        ws, ptr, need = self._workspace(batch, "gemm")
        _call(self.device, _lib().aqlm_i8_gemm, self._ref, ctypes.byref(xs), y.data_ptr(),
              I8_TYPES[dtype], ptr, need)
        return y

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y = Q(x) . W^T, x [batch, in] float16 or bfloat16 quantised token by token on the way."""
        self._check_half(x, "x", self.in_features)
        if x.requires_grad and torch.is_grad_enabled():
            return _record(lambda xs: [self.forward(xs[0])], (self,), (x,), out)[0]
        batch = x.shape[0]
        y = _output(out, (batch, self.out_features), x.dtype, self.device)
        ws, ptr, need = self._workspace(batch, "gemm_quant")
        _call(self.device, _lib().aqlm_i8_gemm_quant, self._ref, x.data_ptr(), batch, y.data_ptr(),
              I8_TYPES[x.dtype], ptr, need)
        return y

    def grad_input(self, dy: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """dx = dy . W: the gradient of forward(x) with respect to x, straight through the
        quantisation. Not recorded by autograd itself."""
        self._check_half(dy, "dy", self.out_features)
        batch = dy.shape[0]
        dx = _output(out, (batch, self.in_features), dy.dtype, self.device)
        ws, ptr, need = self._workspace(batch, "grad_input")
        _call(self.device, _lib().aqlm_i8_grad_input, self._ref, dy.data_ptr(), batch, dx.data_ptr(),
              I8_TYPES[dy.dtype], ptr, need)
        return dx


class _RecordedGated(torch.autograd.Function):
    """A gated block, and for backward its gradient from the saved products."""

    @staticmethod
    def forward(ctx, block, x):
        n, step = block._saved_floats(x.shape[0])
        saved = torch.empty(n, dtype=torch.float32, device=block.device)  # g, then u
        ctx.block = block
        ctx.save_for_backward(saved)
        return block._run(x, None, saved.data_ptr(), saved.data_ptr() + 4 * step)

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        dh = dh.contiguous()
        if dh.data_ptr() % 16:  # a part of a larger gradient
            dh = dh.clone()
        (saved,) = ctx.saved_tensors
        block = ctx.block
        _, step = block._saved_floats(dh.shape[0])
        return None, block._back(dh, saved.data_ptr(), saved.data_ptr() + 4 * step, None)


class I8Gated(_Workspaces):
    """The first half of a gated feed-forward block: h = act(gate(x)) * up(x).

    gate and up are I8Layers of the same sizes, activation "silu", "gelu" or
    "gelu_tanh". x is quantised once for both; both products, the activation
    and their product are one kernel and round once."""

    def __init__(self, gate: I8Layer, up: I8Layer, activation: str = "silu"):
        self._act = _check_act(activation)
        if (gate.out_features, gate.in_features, gate.device) != (up.out_features, up.in_features, up.device):
            raise ValueError("gate and up must have the same sizes and device")
        self.gate, self.up, self.activation = gate, up, activation
        self.out_features, self.in_features, self.device = gate.out_features, gate.in_features, gate.device
        super().__init__(gate._ref, up._ref)

    def _saved_floats(self, batch: int) -> Tuple[int, int]:
        """(floats of g and u in one allocation, where u begins: at a multiple of 16 bytes)."""
        step = (batch * self.out_features + 3) // 4 * 4
        return step + batch * self.out_features, step

    def _run(self, x: torch.Tensor, out: Optional[torch.Tensor], g: Optional[int], u: Optional[int]) -> torch.Tensor:
        batch = x.shape[0]
        h = _output(out, (batch, self.out_features), x.dtype, self.device)
        ws, ptr, need = self._workspace(batch, "gated")
        _call(self.device, _lib().aqlm_i8_gated, self.gate._ref, self.up._ref, x.data_ptr(), batch, self._act,
              h.data_ptr(), g, u, I8_TYPES[x.dtype], ptr, need)
        return h

    def _back(self, dh: torch.Tensor, g: int, u: int, out: Optional[torch.Tensor]) -> torch.Tensor:
        batch = dh.shape[0]
        dx = _output(out, (batch, self.in_features), dh.dtype, self.device)
        ws, ptr, need = self._workspace(batch, "gated_grad")
        _call(self.device, _lib().aqlm_i8_gated_grad, self.gate._ref, self.up._ref, g, u, dh.data_ptr(), batch,
              self._act, dx.data_ptr(), I8_TYPES[dh.dtype], ptr, need)
        return dx

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """h = act(Q(x) . gate^T) * (Q(x) . up^T), x [batch, in] float16 or bfloat16."""
        self._check_half(x, "x", self.in_features)
        if x.requires_grad and torch.is_grad_enabled():
            if out is not None:
                raise ValueError("out takes no part in autograd: x must not require a gradient")
            return _RecordedGated.apply(self, x)
        return self._run(x, out, None, None)

    def forward_saving(self, x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """(h, g, u): forward's result and the float32 products [batch, out] that grad_input takes.
        Not recorded by autograd itself."""
        self._check_half(x, "x", self.in_features)
        g = torch.empty((x.shape[0], self.out_features), dtype=torch.float32, device=self.device)
        u = torch.empty_like(g)
        return self._run(x, None, g.data_ptr(), u.data_ptr()), g, u

    def grad_input(self, dh: torch.Tensor, g: torch.Tensor, u: torch.Tensor,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """dx = (dh u act'(g)) . gate + (dh act(g)) . up: the gradient of forward(x) with respect
        to x, straight through the quantisation, from forward_saving's g and u."""
        self._check_half(dh, "dh", self.out_features)
        for t, what in ((g, "g"), (u, "u")):
            _check_dense(t, what, _FLOAT, dh.shape)
            if t.device != self.device:
                raise ValueError(f"{what} must be on the layer's device")
        return self._back(dh, g.data_ptr(), u.data_ptr(), out)
