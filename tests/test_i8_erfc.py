"""The fitted e^(t^2) erfc(t) behind the int8 blocks' GELU: the coefficients of csrc/i8_device.hpp, evaluated here."""
import os
import re

import numpy as np
import torch

from additive_codebook_matmul_amd import build

FAR = 10.3            # e^(-t^2) is below float32's smallest number from 10.16 on


def _coefficients():
    """Of P, highest power first, as float32."""
    with open(os.path.join(build.CSRC, "i8_device.hpp")) as f:
        body = re.search(r"float scaled_erfc\(float t\) \{(.*?)\n\}", f.read(), re.S).group(1)
    first = re.findall(r"float p = (-?[\d.]+)f;", body)
    rest = re.findall(r"__builtin_fmaf\(p, y, (-?[\d.]+)f\)", body)
    assert len(first) == 1 and len(rest) == 8 and "__builtin_fmaf(0.5f, t, 1.f)" in body
    return [np.float32(c) for c in first + rest]


def _points():
    t = np.concatenate([np.linspace(0, FAR, 200001), np.exp(np.linspace(-40, np.log(FAR), 50001))])
    return t[t <= FAR].astype(np.float32)


def _off(values, t):
    want = torch.special.erfcx(torch.from_numpy(t.astype(np.float64))).numpy()
    return np.abs(values.astype(np.float64) / want - 1).max() * 2.0 ** 24


def test_the_interval_covers_the_function_s_use():
    assert np.float32(np.exp(-FAR * FAR)) == 0


def test_coefficients():
    t = _points()
    y = 1 / (1 + t.astype(np.float64) / 2)
    p = np.zeros_like(y)
    for c in _coefficients():
        p = p * y + float(c)
    assert _off(p * y, t) <= 1.5


def test_float32_operations():
    """Each operation rounded once, with a reciprocal that is exact, a unit too large and a unit too small."""
    t = _points()

    def fma(a, b, c):
        return (a.astype(np.float64) * b.astype(np.float64) + float(c)).astype(np.float32)
    d = fma(t, np.full_like(t, 0.5), 1.0)
    near = (1 / d.astype(np.float64)).astype(np.float32)
    for y in (near, np.nextafter(near, np.float32(2)), np.nextafter(near, np.float32(0))):
        p = np.full_like(y, _coefficients()[0])
        for c in _coefficients()[1:]:
            p = fma(p, y, c)
        assert _off((p * y).astype(np.float32), t) <= 9


def test_far_beyond_it():
    t = np.exp(np.linspace(np.log(FAR), 80, 20001))
    y = 1 / (1 + t / 2)
    p = np.zeros_like(y)
    for c in _coefficients():
        p = p * y + float(c)
    assert _off(p * y, t) <= 2 ** 10
