"""The int8 entry points on the host: declared, exported, and refusing bad arguments before
anything is launched (no GPU needed); the oracle's pins."""
import ctypes
import os
import re
from fractions import Fraction

import numpy as np
import pytest
import torch

import additive_codebook_matmul_amd as pkg
from additive_codebook_matmul_amd import i8
from oracle import i8_oracle as IO

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, MISALIGNED = 0x10000, 0x10008
NULL, SHAPE, ALIGN, BATCH, WORKSPACE, TYPE = 1, 2, 4, 5, 7, 9
BIG = 1 << 40


def M(rows=64, cols=128, codes=FAKE, scales=FAKE + 0x100000):
    return ctypes.byref(i8.I8MatrixStruct(rows, cols, codes, scales))


BAD_MATRICES = [(None, NULL), (M(rows=0), SHAPE), (M(rows=-1), SHAPE), (M(rows=(1 << 21) + 1), SHAPE),
                (M(cols=0), SHAPE), (M(cols=8), SHAPE), (M(cols=100), SHAPE), (M(cols=1 << 17), SHAPE),
                (M(codes=0), NULL), (M(scales=0), NULL), (M(codes=MISALIGNED), ALIGN),
                (M(scales=MISALIGNED), ALIGN)]


def test_header_symbols_exported():
    text = open(os.path.join(ROOT, "include", "aqlm_i8.h")).read()
    declared = set(re.findall(r"AQLM_API\s+[\w\s\*]*?\b(aqlm_\w+)\s*\(", text))
    assert declared == set(i8.I8_SYMBOLS)
    for name in declared:
        assert hasattr(i8._lib(), name), name
    assert ctypes.sizeof(i8.I8MatrixStruct) == 32
    for name in ("I8Layer", "I8Gated", "i8_quantize", "i8_dequant"):
        assert name in pkg.__all__ and hasattr(pkg, name)


def test_quantize_refusals():
    f = i8._lib().aqlm_i8_quantize   # x, type, rows, cols, codes, scales, stream
    assert f(FAKE, 3, 4, 64, FAKE, FAKE, None) == TYPE
    assert f(FAKE, -1, 4, 64, FAKE, FAKE, None) == TYPE
    for rows, cols in ((-1, 64), (4, 0), (4, 8), (4, 17), (4, 40), (4, -16), (1 << 31, 16),
                       (1 << 20, 1 << 21), (4, 1 << 31)):
        assert f(FAKE, 0, rows, cols, FAKE, FAKE, None) == SHAPE, (rows, cols)
    assert f(None, 0, 4, 64, FAKE, FAKE, None) == NULL
    assert f(FAKE, 0, 4, 64, None, FAKE, None) == NULL
    assert f(FAKE, 0, 4, 64, FAKE, None, None) == NULL
    for k in (0, 4, 5):
        args = [FAKE, 0, 4, 64, FAKE, FAKE, None]
        args[k] = MISALIGNED
        assert f(*args) == ALIGN
    assert f(None, 0, 0, 64, None, None, None) == 0          # no rows: no-op


def test_dequant_refusals():
    f = i8._lib().aqlm_i8_dequant    # m, type, W, stream
    assert f(None, 0, FAKE, None) == NULL
    assert f(M(), 3, FAKE, None) == TYPE
    assert f(M(cols=40), 0, FAKE, None) == SHAPE
    assert f(M(rows=-1), 0, FAKE, None) == SHAPE
    assert f(M(codes=0), 0, FAKE, None) == NULL
    assert f(M(scales=MISALIGNED), 0, FAKE, None) == ALIGN
    assert f(M(), 0, None, None) == NULL
    assert f(M(), 0, MISALIGNED, None) == ALIGN
    assert f(M(rows=0, codes=0, scales=0), 0, None, None) == 0


@pytest.mark.parametrize("name", ["aqlm_i8_gemm_quant", "aqlm_i8_grad_input"])
def test_product_refusals(name):
    f = getattr(i8._lib(), name)     # W, x, batch, y, type, ws, bytes, stream
    for bad, status in BAD_MATRICES:
        assert f(bad, FAKE, 1, FAKE, 0, FAKE, BIG, None) == status
    assert f(M(), FAKE, 1, FAKE, 2, FAKE, BIG, None) == TYPE     # float32 is not a product type
    assert f(M(), FAKE, 1, FAKE, -1, FAKE, BIG, None) == TYPE
    assert f(M(), FAKE, -1, FAKE, 0, FAKE, BIG, None) == BATCH
    assert f(M(), FAKE, (1 << 21) + 1, FAKE, 0, FAKE, BIG, None) == BATCH
    assert f(M(), None, 1, FAKE, 0, FAKE, BIG, None) == NULL
    assert f(M(), FAKE, 1, None, 0, FAKE, BIG, None) == NULL
    assert f(M(), MISALIGNED, 1, FAKE, 0, FAKE, BIG, None) == ALIGN
    assert f(M(), FAKE, 1, MISALIGNED, 0, FAKE, BIG, None) == ALIGN
    assert f(M(), None, 0, None, 0, None, 0, None) == 0


def test_gemm_refusals():
    f = i8._lib().aqlm_i8_gemm       # W, x, y, type, ws, bytes, stream
    X = lambda **k: M(**{"rows": 3, **k})  # noqa: E731
    for bad, status in BAD_MATRICES:
        assert f(bad, X(), FAKE, 0, FAKE, BIG, None) == status
    assert f(M(), None, FAKE, 0, FAKE, BIG, None) == NULL
    assert f(M(), X(cols=144), FAKE, 0, FAKE, BIG, None) == SHAPE
    assert f(M(), X(rows=-1), FAKE, 0, FAKE, BIG, None) == SHAPE
    assert f(M(), X(rows=(1 << 21) + 1), FAKE, 0, FAKE, BIG, None) == SHAPE
    assert f(M(), X(scales=0), FAKE, 0, FAKE, BIG, None) == NULL
    assert f(M(), X(codes=MISALIGNED), FAKE, 0, FAKE, BIG, None) == ALIGN
    assert f(M(), X(), FAKE, 2, FAKE, BIG, None) == TYPE
    assert f(M(), X(), None, 0, FAKE, BIG, None) == NULL
    assert f(M(), X(), MISALIGNED, 0, FAKE, BIG, None) == ALIGN
    assert f(M(), X(rows=0, codes=0, scales=0), None, 0, None, 0, None) == 0


def test_gated_refusals():
    f = i8._lib().aqlm_i8_gated      # gate, up, x, batch, act, h, g, u, type, ws, bytes, stream
    ok = [M(), M(), FAKE, 1, 0, FAKE, None, None, 0, FAKE, BIG, None]

    def given(**change):
        args = list(ok)
        for k, v in change.items():
            args[int(k[1:])] = v
        return f(*args)
    for bad, status in BAD_MATRICES:
        assert given(_0=bad) == status and given(_1=bad) == status
    assert given(_1=M(rows=65)) == SHAPE and given(_1=M(cols=144)) == SHAPE
    assert given(_4=3) == TYPE and given(_4=-1) == TYPE and given(_8=2) == TYPE
    assert given(_3=-1) == BATCH and given(_3=(1 << 21) + 1) == BATCH
    assert given(_2=None) == NULL and given(_5=None) == NULL
    assert given(_6=FAKE) == NULL and given(_7=FAKE) == NULL     # one of the two alone
    assert given(_2=MISALIGNED) == ALIGN and given(_5=MISALIGNED) == ALIGN
    assert given(_6=MISALIGNED, _7=FAKE) == ALIGN and given(_6=FAKE, _7=MISALIGNED) == ALIGN
    assert given(_3=0, _2=None, _5=None, _9=None, _10=0) == 0


def test_gated_grad_refusals():
    f = i8._lib().aqlm_i8_gated_grad  # gate, up, g, u, dh, batch, act, dx, type, ws, bytes, stream
    ok = [M(), M(), FAKE, FAKE, FAKE, 1, 0, FAKE, 0, FAKE, BIG, None]

    def given(**change):
        args = list(ok)
        for k, v in change.items():
            args[int(k[1:])] = v
        return f(*args)
    for bad, status in BAD_MATRICES:
        assert given(_0=bad) == status and given(_1=bad) == status
    assert given(_1=M(rows=63)) == SHAPE
    assert given(_6=3) == TYPE and given(_6=-1) == TYPE and given(_8=2) == TYPE
    assert given(_5=-1) == BATCH and given(_5=(1 << 21) + 1) == BATCH
    for k in ("_2", "_3", "_4", "_7"):
        assert given(**{k: None}) == NULL and given(**{k: MISALIGNED}) == ALIGN
    assert given(_5=0, _2=None, _3=None, _4=None, _7=None, _9=None, _10=0) == 0


@pytest.mark.parametrize("op", ["gemm", "gemm_quant", "grad_input", "gated", "gated_grad"])
def test_workspace_size(op):
    lib = i8._lib()
    f, two = getattr(lib, f"aqlm_i8_{op}_workspace_size"), op.startswith("gated")
    n = ctypes.c_int64(-1)

    def size(w, batch, out=ctypes.byref(n)):
        return f(w, w, batch, out) if two else f(w, batch, out)
    assert size(M(), 1, None) == NULL
    assert size(None, 1) == NULL and n.value == 0
    assert size(M(), -1) == BATCH and n.value == 0
    assert size(M(cols=40), 1) == SHAPE
    assert size(M(), 0) == 0 and n.value == 0
    if two:
        assert f(M(), M(rows=65), 1, ctypes.byref(n)) == SHAPE
    for rows, cols in ((1, 16), (4096, 11008), (11008, 4096), (300, 1 << 15)):
        for batch in (1, 5, 17, 77, 128, 300, 2048):
            w = M(rows, cols)
            assert size(w, batch) == 0
            need = n.value
            assert 0 <= need <= 1 << 30
            calls = {"gemm": lambda ws, b: lib.aqlm_i8_gemm(w, M(batch, cols), FAKE, 0, ws, b, None),
                     "gemm_quant": lambda ws, b: lib.aqlm_i8_gemm_quant(w, FAKE, batch, FAKE, 0, ws, b, None),
                     "grad_input": lambda ws, b: lib.aqlm_i8_grad_input(w, FAKE, batch, FAKE, 0, ws, b, None),
                     "gated": lambda ws, b: lib.aqlm_i8_gated(w, w, FAKE, batch, 0, FAKE, None, None, 0, ws, b, None),
                     "gated_grad": lambda ws, b: lib.aqlm_i8_gated_grad(w, w, FAKE, FAKE, FAKE, batch, 0, FAKE, 0,
                                                                        ws, b, None)}
            if need:  # too little is refused before anything is launched
                assert calls[op](None, need) == NULL
                assert calls[op](MISALIGNED, need) == ALIGN
                assert calls[op](FAKE, need - 1) == WORKSPACE


def test_binding_refuses_host_and_wrong_tensors():
    codes = torch.zeros((4, 32), dtype=torch.int8)
    scales = torch.zeros(4)
    with pytest.raises(ValueError):
        i8.I8Layer(codes, scales)
    with pytest.raises(ValueError):
        i8.i8_quantize(torch.zeros((4, 64)))
    with pytest.raises(ValueError):
        i8.i8_dequant(codes, scales)
    with pytest.raises(ValueError, match="activation"):
        i8.I8Gated(None, None, "relu")


# --- the oracle, pinned to hand-worked values and exact fractions -------------
def test_oracle_codes():
    x = np.zeros((4, 16))
    x[0, :4] = [127, 0.5, 1.5, -2.5]                 # ties to even
    x[1, :3] = [-254, 1, 3]                          # 127 x / 254 = x / 2
    x[2, :2] = [np.inf, 1]
    codes, scales = IO.quantize(x)
    assert codes[0, :4].tolist() == [127, 0, 2, -2] and scales[0] == 1
    assert codes[1, :3].tolist() == [-127, 0, 2] and scales[1] == 2
    assert not codes[2:].any() and np.isnan(scales[2]) and scales[3] == 0


def test_oracle_codes_against_fractions():
    rng = np.random.default_rng(1)
    for dtype in (np.float16, np.float32):
        x = (rng.standard_normal((6, 64)) * np.exp2(rng.integers(-12, 12, (6, 1)))).astype(dtype)
        x[:3] = np.round(x[:3] * 4) / 4              # many ties
        x[0, 0], x[1, 0] = 127, 254
        codes, scales = IO.quantize(x.astype(np.float64))
        for r in range(6):
            top = max(abs(Fraction(float(v))) for v in x[r])
            if top == 0:
                assert scales[r] == 0 and not codes[r].any()
                continue
            for c in range(64):
                assert codes[r, c] == round(Fraction(float(x[r, c])) * 127 / top)   # ties to even
            assert abs(Fraction(float(scales[r])) - top / 127) <= top / 127 / 2 ** 24


def test_oracle_products_and_activations():
    s = IO.sums(np.array([[1, -2]], np.int8), np.array([[3, 4], [-128, 127]], np.int8))
    assert s.tolist() == [[-5, -382]]
    assert IO.value(s, np.array([2, .5]), np.array([4.0])).tolist() == [[-40, -764]]
    for name in IO.ACTIVATIONS:
        a, d = IO.act(np.array([0.0, 40.0, -40.0]), name)
        assert a[0] == 0 and d[0] == 0.5 and a[1] == 40 and abs(d[1] - 1) < 1e-12
        assert abs(a[2]) < 1e-12 and abs(d[2]) < 1e-12
        z, e = np.linspace(-4, 4, 41), 1e-5
        slope = (IO.act(z + e, name)[0] - IO.act(z - e, name)[0]) / (2 * e)
        assert np.abs(slope - IO.act(z, name)[1]).max() < 1e-9
    assert abs(IO.act(np.array([1.0]), "silu")[0][0] - 0.7310585786300049) < 1e-15
    assert abs(IO.act(np.array([1.0]), "gelu")[0][0] - 0.8413447460685429) < 1e-15
    assert abs(IO.act(np.array([1.0]), "gelu_tanh")[0][0] - 0.8411919906082768) < 1e-15
    t, b = IO.back(np.array([[1.0, -2.0]]), np.array([[3, 4], [5, -6]], np.int8))
    assert t.tolist() == [[-7, 16]] and b.tolist() == [[13, 16]]
