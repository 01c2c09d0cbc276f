"""CPU oracle of the 8-bit integer (int8) operators.

TEST INFRASTRUCTURE ONLY (numpy, no code shared with the library). The rules are
those of include/aqlm_i8.h; everything is evaluated in float64 or in whole
numbers, and rounded to float32 only where the header says that a value is one.
"""
from __future__ import annotations

import math

import numpy as np

ACTIVATIONS = ("silu", "gelu", "gelu_tanh")


def quantize(x: np.ndarray):
    """(codes int8 [rows, cols], scales float32 [rows]) of a float64 matrix of float32 values.

    127 x is exact in float64 and the quotient rounded once, which keeps a tie a
    tie and moves nothing onto or across one: a quotient that is no tie is at
    least 2^-34 away from it."""
    top = np.abs(x).max(axis=1, keepdims=True)
    good = np.isfinite(x).all(axis=1, keepdims=True)
    safe = np.where(good & (top > 0), top, 1.0)
    codes = np.where(good, np.rint(np.where(good, x, 0.0) * 127.0 / safe), 0.0)
    with np.errstate(invalid="ignore"):
        scales = np.where(good, top.astype(np.float32) / np.float32(127.0), np.float32(np.nan))
    return codes.astype(np.int8), scales[:, 0].astype(np.float32)


def value(sums: np.ndarray, channel: np.ndarray, token: np.ndarray) -> np.ndarray:
    """float32 products [batch, rows] of exact sums, in the order of the operations."""
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        return (sums.astype(np.float32) * channel[None, :].astype(np.float32)) * token[:, None].astype(np.float32)


def sums(xcodes: np.ndarray, wcodes: np.ndarray) -> np.ndarray:
    """Exact sums of codes [batch, rows] (float64 holds them)."""
    return xcodes.astype(np.float64) @ wcodes.astype(np.float64).T


def act(g: np.ndarray, name: str):
    """(act(g), act'(g)) in float64."""
    g = np.asarray(g, dtype=np.float64)
    with np.errstate(over="ignore"):
        if name == "silu":
            s = 1.0 / (1.0 + np.exp(-g))
            return g * s, s * (1.0 + g * (1.0 - s))
        if name == "gelu":
            phi = 0.5 * np.vectorize(math.erfc)(-g / math.sqrt(2.0))
            return g * phi, phi + g * np.exp(-g * g / 2.0) / math.sqrt(2.0 * math.pi)
        c, a = 2.0 * math.sqrt(2.0 / math.pi), 0.044715
        s = 1.0 / (1.0 + np.exp(-c * (g + a * g ** 3)))
        return g * s, s + g * s * (1.0 - s) * c * (1.0 + 3.0 * a * g * g)


def gated_terms(g, u, dh, wg, wu, name):
    """The two gradients times channel scales, [batch, rows] each, in float64."""
    a, slope = act(g, name)
    return dh * u * slope * wg[None, :], dh * a * wu[None, :]


def back(terms, codes):
    """(sum over rows of terms . codes, sum |terms codes|) in float64."""
    c = codes.astype(np.float64)
    return terms @ c, np.abs(terms) @ np.abs(c)
