"""The microscaled entry points on the host: declared, exported, and refusing bad
arguments before anything is launched (no GPU needed); the oracle's pins."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import additive_codebook_matmul_amd as pkg
from additive_codebook_matmul_amd import _lib, mx
from oracle import mx_oracle as MO

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, MISALIGNED = 0x10000, 0x10008
NULL, SHAPE, ALIGN, BATCH, WORKSPACE, TYPE = 1, 2, 4, 5, 7, 9


def M(rows=64, cols=128, codes=FAKE, scales=FAKE + 0x100000):
    return ctypes.byref(mx.MxMatrixStruct(rows, cols, codes, scales))


def test_header_symbols_exported():
    text = open(os.path.join(ROOT, "include", "aqlm_mx.h")).read()
    declared = set(re.findall(r"AQLM_API\s+[\w\s\*]*?\b(aqlm_\w+)\s*\(", text))
    assert declared == set(mx.MX_SYMBOLS)
    for name in declared:
        assert hasattr(mx._lib(), name), name
    assert ctypes.sizeof(mx.MxMatrixStruct) == 32
    assert "element type" in _lib.status_string(TYPE)
    for name in ("MxLayer", "mx_quantize", "mx_dequant", "mx_gemv_batched"):
        assert name in pkg.__all__ and hasattr(pkg, name)


def test_quantize_refusals():
    f = mx._lib().aqlm_mx_quantize   # x, type, rows, cols, rule, codes, scales, stream
    assert f(FAKE, 3, 4, 64, 0, FAKE, FAKE, None) == TYPE
    assert f(FAKE, -1, 4, 64, 0, FAKE, FAKE, None) == TYPE
    assert f(FAKE, 0, 4, 64, 2, FAKE, FAKE, None) == TYPE
    for rows, cols in ((-1, 64), (4, 0), (4, 16), (4, 33), (4, 48), (4, -32), (1 << 31, 32),
                       (1 << 20, 1 << 21), (4, 1 << 31)):
        assert f(FAKE, 0, rows, cols, 0, FAKE, FAKE, None) == SHAPE, (rows, cols)
    assert f(None, 0, 4, 64, 0, FAKE, FAKE, None) == NULL
    assert f(FAKE, 0, 4, 64, 0, None, FAKE, None) == NULL
    assert f(FAKE, 0, 4, 64, 0, FAKE, None, None) == NULL
    assert f(MISALIGNED, 0, 4, 64, 0, FAKE, FAKE, None) == ALIGN
    assert f(FAKE, 0, 4, 64, 0, MISALIGNED, FAKE, None) == ALIGN
    assert f(FAKE, 0, 4, 64, 0, FAKE, MISALIGNED, None) == ALIGN
    assert f(None, 0, 0, 64, 0, None, None, None) == 0          # no rows: no-op


def test_dequant_refusals():
    f = mx._lib().aqlm_mx_dequant    # m, type, W, stream
    assert f(None, 0, FAKE, None) == NULL
    assert f(M(), 3, FAKE, None) == TYPE
    assert f(M(cols=40), 0, FAKE, None) == SHAPE
    assert f(M(rows=-1), 0, FAKE, None) == SHAPE
    assert f(M(codes=0), 0, FAKE, None) == NULL
    assert f(M(scales=MISALIGNED), 0, FAKE, None) == ALIGN
    assert f(M(), 0, None, None) == NULL
    assert f(M(), 0, MISALIGNED, None) == ALIGN
    assert f(M(rows=0, codes=0, scales=0), 0, None, None) == 0


@pytest.mark.parametrize("name", ["aqlm_mx_gemm", "aqlm_mx_grad_input"])
def test_product_refusals(name):
    f = getattr(mx._lib(), name)     # W, x, batch, y, type, ws, bytes, stream
    big = 1 << 40
    assert f(None, FAKE, 1, FAKE, 0, FAKE, big, None) == NULL
    assert f(M(rows=0), FAKE, 1, FAKE, 0, FAKE, big, None) == SHAPE
    assert f(M(rows=(1 << 21) + 1), FAKE, 1, FAKE, 0, FAKE, big, None) == SHAPE
    assert f(M(cols=(1 << 21) + 32), FAKE, 1, FAKE, 0, FAKE, big, None) == SHAPE
    assert f(M(cols=100), FAKE, 1, FAKE, 0, FAKE, big, None) == SHAPE
    assert f(M(codes=0), FAKE, 1, FAKE, 0, FAKE, big, None) == NULL
    assert f(M(codes=MISALIGNED), FAKE, 1, FAKE, 0, FAKE, big, None) == ALIGN
    assert f(M(), FAKE, 1, FAKE, 2, FAKE, big, None) == TYPE     # float32 is not a product type
    assert f(M(), FAKE, -1, FAKE, 0, FAKE, big, None) == BATCH
    assert f(M(), FAKE, (1 << 21) + 1, FAKE, 0, FAKE, big, None) == BATCH
    assert f(M(), None, 1, FAKE, 0, FAKE, big, None) == NULL
    assert f(M(), FAKE, 1, None, 0, FAKE, big, None) == NULL
    assert f(M(), MISALIGNED, 1, FAKE, 0, FAKE, big, None) == ALIGN
    assert f(M(), FAKE, 1, MISALIGNED, 0, FAKE, big, None) == ALIGN
    assert f(M(), None, 0, None, 0, None, 0, None) == 0


def test_gemm_mx_refusals():
    f = mx._lib().aqlm_mx_gemm_mx    # W, x, y, type, ws, bytes, stream
    big = 1 << 40
    X = lambda **k: M(**{"rows": 3, **k})  # noqa: E731
    assert f(None, X(), FAKE, 0, FAKE, big, None) == NULL
    assert f(M(), None, FAKE, 0, FAKE, big, None) == NULL
    assert f(M(), X(cols=160), FAKE, 0, FAKE, big, None) == SHAPE
    assert f(M(), X(rows=-1), FAKE, 0, FAKE, big, None) == SHAPE
    assert f(M(), X(scales=0), FAKE, 0, FAKE, big, None) == NULL
    assert f(M(), X(codes=MISALIGNED), FAKE, 0, FAKE, big, None) == ALIGN
    assert f(M(), X(), FAKE, 2, FAKE, big, None) == TYPE
    assert f(M(), X(), None, 0, FAKE, big, None) == NULL
    assert f(M(), X(), MISALIGNED, 0, FAKE, big, None) == ALIGN
    assert f(M(), X(rows=0, codes=0, scales=0), None, 0, None, 0, None) == 0


def test_gemm_quant_refusals():
    f = mx._lib().aqlm_mx_gemm_quant  # W, x, batch, rule, y, type, ws, bytes, stream
    size = mx._lib().aqlm_mx_gemm_quant_workspace_size
    big = 1 << 40
    assert f(None, FAKE, 1, 0, FAKE, 0, FAKE, big, None) == NULL
    assert f(M(rows=0), FAKE, 1, 0, FAKE, 0, FAKE, big, None) == SHAPE
    assert f(M(cols=100), FAKE, 1, 0, FAKE, 0, FAKE, big, None) == SHAPE
    assert f(M(), FAKE, 1, 0, FAKE, 2, FAKE, big, None) == TYPE
    assert f(M(), FAKE, 1, 2, FAKE, 0, FAKE, big, None) == TYPE
    assert f(M(), FAKE, 1, -1, FAKE, 0, FAKE, big, None) == TYPE
    assert f(M(), FAKE, -1, 0, FAKE, 0, FAKE, big, None) == BATCH
    assert f(M(), FAKE, (1 << 21) + 1, 0, FAKE, 0, FAKE, big, None) == BATCH
    assert f(M(), None, 1, 0, FAKE, 0, FAKE, big, None) == NULL
    assert f(M(), FAKE, 1, 0, None, 0, FAKE, big, None) == NULL
    assert f(M(), MISALIGNED, 1, 0, FAKE, 0, FAKE, big, None) == ALIGN
    assert f(M(), FAKE, 1, 0, MISALIGNED, 0, FAKE, big, None) == ALIGN
    assert f(M(), None, 0, 0, None, 0, None, 0, None) == 0
    n, own = ctypes.c_int64(-1), ctypes.c_int64(-1)
    for rows, cols, batch in ((64, 32, 7), (4096, 11008, 77), (300, 1 << 15, 300)):
        assert size(M(rows, cols), batch, ctypes.byref(n)) == 0
        assert mx._lib().aqlm_mx_gemm_mx_workspace_size(M(rows, cols), batch, ctypes.byref(own)) == 0
        assert n.value >= batch * cols * 17 // 32 + own.value
        for ws, given, st in ((None, n.value, NULL), (MISALIGNED, n.value, ALIGN),
                              (FAKE, n.value - 1, WORKSPACE)):
            assert f(M(rows, cols), FAKE, batch, 0, FAKE, 0, ws, given, None) == st


def test_gemv_batched_refusals():
    f = mx._lib().aqlm_mx_gemv_batched  # W, x, y, n, batch, type, stream
    ok = mx.MxMatrixStruct(64, 128, FAKE, FAKE)
    two = (mx.MxMatrixStruct * 2)(ok, mx.MxMatrixStruct(64, 100, FAKE, FAKE))
    good = (mx.MxMatrixStruct * 2)(ok, ok)
    p = (ctypes.c_void_p * 2)(FAKE, FAKE + 0x1000)
    bad = (ctypes.c_void_p * 2)(FAKE, MISALIGNED)
    none = (ctypes.c_void_p * 2)(FAKE, 0)
    assert f(good, p, p, -1, 1, 0, None) == SHAPE
    assert f(good, p, p, 4097, 1, 0, None) == SHAPE
    assert f(good, p, p, 2, 9, 0, None) == BATCH
    assert f(good, p, p, 2, -1, 0, None) == BATCH
    assert f(good, p, p, 2, 1, 2, None) == TYPE
    assert f(None, p, p, 2, 1, 0, None) == NULL
    assert f(good, None, p, 2, 1, 0, None) == NULL
    assert f(two, p, p, 2, 1, 0, None) == SHAPE    # the second layer: nothing is launched
    assert f(good, bad, p, 2, 1, 0, None) == ALIGN
    assert f(good, p, none, 2, 1, 0, None) == NULL
    assert f(None, None, None, 0, 1, 0, None) == 0
    assert f(None, None, None, 2, 0, 0, None) == 0


@pytest.mark.parametrize("op", ["gemm", "gemm_mx", "grad_input"])
def test_workspace_size(op):
    f = getattr(mx._lib(), f"aqlm_mx_{op}_workspace_size")
    n = ctypes.c_int64(-1)
    assert f(M(), 1, None) == NULL
    assert f(None, 1, ctypes.byref(n)) == NULL and n.value == 0
    assert f(M(), -1, ctypes.byref(n)) == BATCH and n.value == 0
    assert f(M(cols=48), 1, ctypes.byref(n)) == SHAPE
    assert f(M(), 0, ctypes.byref(n)) == 0 and n.value == 0
    for rows, cols in ((1, 32), (4096, 11008), (11008, 4096), (300, 1 << 15)):
        for batch in (1, 5, 17, 77, 128, 300, 2048):
            assert f(M(rows, cols), batch, ctypes.byref(n)) == 0
            assert 0 <= n.value <= 1 << 30
            if n.value:  # too little is refused before anything is launched
                need, big = n.value, getattr(mx._lib(), f"aqlm_mx_{op}")
                for ws, given, st in ((None, need, NULL), (MISALIGNED, need, ALIGN),
                                      (FAKE, need - 1, WORKSPACE)):
                    if op == "gemm_mx":
                        assert big(M(rows, cols), M(batch, cols), FAKE, 0, ws, given, None) == st
                    else:
                        assert big(M(rows, cols), FAKE, batch, FAKE, 0, ws, given, None) == st


def test_binding_refuses_host_and_wrong_tensors():
    codes = torch.zeros((4, 32), dtype=torch.uint8)
    scales = torch.zeros((4, 2), dtype=torch.uint8)
    with pytest.raises(ValueError):
        mx.MxLayer(codes, scales)
    with pytest.raises(ValueError):
        mx.mx_quantize(torch.zeros((4, 64)))
    with pytest.raises(ValueError):
        mx.mx_dequant(codes, scales)
    assert mx.mx_gemv_batched([], []) == []
    with pytest.raises(ValueError):
        mx.mx_gemv_batched([], [1])


# --- the oracle, pinned to hand-worked values --------------------------------
def test_oracle_codes_and_packing():
    assert MO.E2M1.tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    assert np.signbit(MO.E2M1[8])
    codes = np.arange(32, dtype=np.uint8)[None] % 16
    assert MO.pack(codes)[0, :3].tolist() == [0x10, 0x32, 0x54]
    assert np.array_equal(MO.unpack(MO.pack(codes)), codes)
    w = MO.dequant(MO.pack(codes), np.array([[129]], np.uint8))     # scale 4
    assert w[0, :8].tolist() == [0, 2, 4, 6, 8, 12, 16, 24]
    assert np.isnan(MO.dequant(MO.pack(codes), np.array([[255]], np.uint8))).all()
    assert MO.scale_value(np.array([0, 127, 254])).tolist() == [2.0 ** -127, 1.0, 2.0 ** 127]


def test_oracle_scales_and_rounding():
    def q(first, rule="floor", rest=0.0):
        x = np.full((1, 32), rest)
        x[0, 0] = first
        codes, s = MO.quantize(x, rule)
        return int(s[0, 0]), int(MO.unpack(codes)[0, 0]), int(MO.unpack(codes)[0, 1])
    assert q(6.0) == (127, 7, 0) and q(4.0) == (127, 6, 0) and q(3.99) == (126, 7, 0)
    assert q(7.9) == (127, 7, 0)                    # clipped to 6
    assert q(7.9, "ceil") == (128, 6, 0)            # 3.95 -> 4
    assert q(6.0, "ceil") == (127, 7, 0) and q(6.01, "ceil") == (128, 5, 0)
    assert q(-5.0) == (127, 14, 0)                  # tie between 4 and 6: the even code, 4
    assert q(6.0, rest=0.25)[2] == 0 and q(6.0, rest=0.75)[2] == 2   # ties to even
    assert q(6.0, rest=1.25)[2] == 2 and q(6.0, rest=1.75)[2] == 4
    assert q(6.0, rest=2.5)[2] == 4 and q(6.0, rest=3.5)[2] == 6
    assert q(0.0) == (127, 0, 0) and q(-0.0) == (127, 8, 0)
    assert q(np.nan) == (255, 0, 0) and q(np.inf, rest=1.0) == (255, 0, 0)
    assert q(2.0 ** -149)[0] == 0 and q(2.0 ** -125)[:2] == (0, 6)


def test_oracle_products():
    x = np.array([[1.0, 2.0], [0.0, -1.0]])
    w = np.array([[3.0, 4.0], [-5.0, 6.0], [0.5, 0.0]])
    assert MO.product(x, w)[0].tolist() == [[11, 7, 0.5], [-4, -6, 0]]
    assert MO.product(x, w)[1].tolist() == [[11, 17, 0.5], [4, 6, 0]]
    assert MO.grad_input(np.array([[1.0, 1.0, 2.0]]), w)[0].tolist() == [[-1, 10]]
