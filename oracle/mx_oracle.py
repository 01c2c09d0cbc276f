"""CPU oracle of the microscaled 4-bit (MXFP4) operators.

TEST INFRASTRUCTURE ONLY (numpy, no code shared with the library). Values and
rules are those of the "OCP Microscaling Formats (MX) Specification" v1.0,
MXFP4: blocks of 32 E2M1 values with one E8M0 power of two, plus the rules
that the specification leaves open (the choice of scale, zeros, non-finite
inputs) as include/aqlm_mx.h states them. Everything is evaluated in float64,
which holds every operand exactly.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([E2M1, -E2M1])


def pack(codes: np.ndarray) -> np.ndarray:
    """[rows, cols] 4-bit codes -> [rows, cols/2] bytes, the even column low."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    out = np.empty((packed.shape[0], packed.shape[1] * 2), dtype=np.uint8)
    out[:, 0::2] = packed & 15
    out[:, 1::2] = packed >> 4
    return out


def scale_value(s: np.ndarray) -> np.ndarray:
    v = np.ldexp(1.0, s.astype(np.int64) - 127)
    return np.where(s == 255, np.nan, v)


def dequant(packed: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 [rows, cols]."""
    return E2M1[unpack(packed)] * np.repeat(scale_value(scales), BLOCK, axis=1)


def scale_bytes(x: np.ndarray, rule: str) -> np.ndarray:
    """E8M0 bytes [rows, cols/32] of a float64 matrix, searched over every power of two."""
    rows, cols = x.shape
    blocks = x.reshape(rows, cols // BLOCK, BLOCK)
    top = np.abs(blocks).max(axis=2)
    out = np.empty(top.shape, dtype=np.uint8)
    powers = np.ldexp(1.0, np.arange(-127, 128))      # bytes 0 .. 254
    for r in range(rows):
        for j in range(cols // BLOCK):
            a = top[r, j]
            if not np.isfinite(blocks[r, j]).all():
                out[r, j] = 255
            elif a == 0:
                out[r, j] = 127
            elif rule == "floor":                     # largest 2^e with 4 * 2^e <= a
                fit = np.nonzero(4 * powers <= a)[0]
                out[r, j] = fit[-1] if len(fit) else 0
            else:                                     # smallest 2^e with a <= 6 * 2^e
                out[r, j] = np.nonzero(a <= 6 * powers)[0][0]
    return out


def quantize(x: np.ndarray, rule: str = "floor"):
    """(packed codes, scale bytes) of a float64 matrix."""
    rows, cols = x.shape
    s = scale_bytes(x, rule)
    v = x / np.repeat(np.where(s == 255, 1.0, scale_value(s)), BLOCK, axis=1)
    a = np.abs(v)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])  # between code c and c + 1
    code = np.zeros(x.shape, dtype=np.uint8)
    for c, m in enumerate(mids):                      # a tie goes to the even code of the two
        code += (a > m) if c % 2 == 0 else (a >= m)
    code |= (np.signbit(x).astype(np.uint8) << 3)
    code[np.repeat(s == 255, BLOCK, axis=1)] = 0
    return pack(code), s


def product(x: np.ndarray, w: np.ndarray):
    """(x . w^T, sum |x w|) in float64."""
    with np.errstate(invalid="ignore", over="ignore"):
        return x @ w.T, np.abs(x) @ np.abs(w).T


def grad_input(dy: np.ndarray, w: np.ndarray):
    """(dy . w, sum |dy w|) in float64."""
    with np.errstate(invalid="ignore", over="ignore"):
        return dy @ w, np.abs(dy) @ np.abs(w)
