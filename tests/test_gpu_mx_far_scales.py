"""The microscaled products and the input gradient with weights at the end of their range."""
import numpy as np
import pytest

from additive_codebook_matmul_amd import MxLayer
from oracle import mx_oracle as MO
from test_gpu_mx import HALVES, dev, rounded, same

pytestmark = pytest.mark.gpu

TERMS = 16  # codes other than zero of a row (a column, in the gradient)


# --- weights at and past the end of bfloat16's range ----------------------------
# bfloat16 holds all of these exactly; 1022 and 65504 are not among its values, so that
# float16's two parts are both at work
ENDS = np.array([1.0, 1022.0, -1022.0, 0.0, 65504.0, -1.0, 2047.0, 2.0 ** -14, np.inf, 3.0, -np.inf])


def huge(lines, length, seed):
    """[lines, length]: every seventh line (and the last) one weight of a block of scale byte 252,
    253 or 254, in one of two places, and nothing else; the others small whole numbers."""
    rng = np.random.default_rng(seed)
    codes = np.zeros((lines, length), dtype=np.uint8)
    codes[np.arange(lines)[:, None], rng.integers(0, length, (lines, TERMS))] = rng.integers(1, 16, (lines, TERMS))
    power = np.full((lines, length), 127)
    places = np.array([length // 3, length - 1])
    codes[:, places] = 2                                   # 1.0
    picked = np.unique(np.r_[np.arange(0, lines, 7), lines - 1])
    at = places[rng.integers(0, 2, len(picked))]
    codes[picked] = 0
    codes[picked, at] = rng.integers(0, 2, len(picked)) * 8 + rng.integers(1, 8, len(picked))
    power[picked, at] = 252 + np.arange(len(picked)) % 3
    return codes, power, places


def _ends(tokens, length, places, seed):
    x = np.random.default_rng(seed).integers(-2, 3, (tokens, length)).astype(np.float64)
    for k, p in enumerate(places):
        x[:, p] = ENDS[(np.arange(tokens) + 4 * k) % len(ENDS)]
        x[np.isinf(x[:, places[0]]), p] = ENDS[1 + k]      # one infinity a token
    return x


def _held(w):
    """float64 weights with magnitudes from 2^128 on as infinities."""
    return np.where(np.abs(w) >= 2.0 ** 128, np.copysign(np.inf, w), w)


def _scales_of(power):
    """One byte a block: the one that differs from 127, where there is one."""
    blocks = power.reshape(power.shape[0], -1, 32)
    top = blocks.max(2)
    return np.where(top == 127, 127, top).astype(np.uint8)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", [(1, 330, 2080), (2, 330, 2080), (7, 330, 2080), (13, 330, 2080),
                                            (100, 1030, 1184), (520, 2085, 4640), (1040, 4100, 1056)])
def test_products_with_infinite_weights(batch, out, n_in, dtype):
    """Magnitudes from 2^128 on are infinities and the others finite, as in a dense product: with an
    activation that is not zero an infinity of its sign, with zero NaN."""
    codes, power, places = huge(out, n_in, batch)
    packed, scales = MO.pack(codes), _scales_of(power)
    w = _held(MO.dequant(packed, scales))
    layer = MxLayer(dev(packed), dev(scales))
    for turn in range(1 if batch > 20 else len(ENDS)):     # every value meets few tokens too
        x = rounded(np.roll(_ends(max(batch, len(ENDS)), n_in, places, 5), turn, axis=0)[:batch], dtype)
        want = rounded(MO.product(x.double().numpy(), w)[0], dtype)
        same(layer.gemm(x.to(DEV)), want)
        if batch <= 8:
            same(layer.gemv(x.to(DEV)), want)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", [(3, 330, 96), (40, 2600, 1056), (300, 4099, 5216), (520, 2085, 4640)])
def test_gradients_with_infinite_weights(batch, out, n_in, dtype):
    codes, power, places = huge(n_in, out, batch)          # lines are columns
    for p in places:                                       # a block of 32 columns has one scale in a row
        for b in range(n_in // 32):
            part = slice(32 * b, 32 * b + 32)
            top = int(power[part, p].max())
            rest = power[part, p] != top
            codes[part, p][rest] = 0
            power[part, p] = top
    packed = MO.pack(np.ascontiguousarray(codes.T))
    scales = np.ascontiguousarray(power.T)[:, ::32].astype(np.uint8)
    w = _held(MO.dequant(packed, scales))
    layer = MxLayer(dev(packed), dev(scales))
    for turn in range(len(ENDS) if batch < 20 else 1):
        dy = rounded(np.roll(_ends(max(batch, len(ENDS)), out, places, 5), turn, axis=0)[:batch], dtype)
        want = rounded(MO.grad_input(dy.double().numpy(), w)[0], dtype)
        same(layer.grad_input(dy.to(DEV)), want)
