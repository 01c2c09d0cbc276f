"""The microscaled products and the input gradient with scales far from 1, exactly.

float16 holds every weight of a block exactly for scale bytes 104 .. 140 alone; a
wavefront (a row, at one or two tokens; a workgroup, in the gradient) that meets another
byte goes on in bfloat16 with the activations split in two. Here single bytes outside that
range lie in the first, a middle, the ninth and the last group of K of some wavefronts'
rows, and others have none, in sizes that choose every kernel, tile shape and split of K,
with ragged rows and with scales that end inside words.

The comparison is exact: rows (columns, in the gradient) are sparse and of three kinds,
each with scales near one power of two, so that every partial sum is a whole multiple of
the kind's unit below 2^24 units, with activations that use all eleven (eight) bits of
their type. Float32 sums are then exact in any order and the result has to be the exact
sum rounded once.
"""
import numpy as np
import pytest
import torch

from additive_codebook_matmul_amd import MxLayer, mx_gemv_batched
from oracle import mx_oracle as MO
from test_gpu_mx import DEV, HALVES, dev, guarded, rounded, same

pytestmark = pytest.mark.gpu

# kinds of rows: usual scale bytes, bytes that float16 cannot take, the unit (half the least scale)
LOW, USUAL, HIGH = 0, 1, 2
NEAR = {LOW: (104, 105), USUAL: (125, 129), HIGH: (137, 140)}
FAR = {LOW: (102, 103), USUAL: (90, 90), HIGH: (141, 142)}
UNIT = np.exp2([102.0 - 128, 125.0 - 128, 137.0 - 128])
TERMS = 16  # codes other than zero of a row (a column, in the gradient), and one in each far block


def _near(kinds, rng):
    low, high = np.array([NEAR[k] for k in range(3)])[kinds].T
    return rng.integers(low, high + 1)


def _top(dtype):
    return 2047 if dtype == torch.float16 else 255


def _integers(rows, cols, dtype, seed):
    top = _top(dtype)
    return np.random.default_rng(seed).integers(-top, top + 1, (rows, cols)).astype(np.float64)


def far_rows(out, n_in, seed):
    """Weights whose rows are of one kind each. Every fifth band of 32 rows has no far scale, the
    others have one in three rows, one of each kind, in a group of K of the band's own."""
    rng = np.random.default_rng(seed)
    nb, groups = n_in // 32, (n_in // 32 + 15) // 16
    kinds = rng.integers(0, 3, out)
    codes = np.zeros((out, n_in), dtype=np.uint8)
    codes[np.arange(out)[:, None], rng.integers(0, n_in, (out, TERMS))] = rng.integers(1, 16, (out, TERMS))
    places = []
    for band in range((out + 31) // 32):
        group = (None, 0, groups // 2, min(8, groups - 1), groups - 1)[band % 5]
        rows = rng.permutation(np.arange(32 * band, min(out, 32 * band + 32)))[:3]
        if group is not None:
            for kind, row in enumerate(rows):
                kinds[row] = kind
                places.append((row, int(rng.integers(16 * group, min(nb, 16 * group + 16))), kind))
    scales = np.empty((out, nb), dtype=np.uint8)
    for b in range(nb):
        scales[:, b] = _near(kinds, rng)
    for row, b, kind in places:
        scales[row, b] = rng.integers(FAR[kind][0], FAR[kind][1] + 1)
        codes[row, 32 * b:32 * b + 32] = 0
        if kind != USUAL:
            codes[row, 32 * b + rng.integers(32)] = rng.integers(1, 16)
    packed = MO.pack(codes)
    w = MO.dequant(packed, scales)
    assert (np.abs(w).sum(1) * 2047 < UNIT[kinds] * 2.0 ** 24).all()
    assert ((w / UNIT[kinds][:, None]) % 1 == 0).all()
    return packed, scales, w


def far_columns(out, n_in, seed):
    """Weights whose blocks of columns are of one kind each; of every four runs of 256 columns one
    has no far scale, the others in the first, a middle and the last 256 rows alone."""
    rng = np.random.default_rng(seed)
    nb, groups = n_in // 32, (out + 255) // 256
    kinds = rng.integers(0, 3, nb)
    codes = np.zeros((out, n_in), dtype=np.uint8)
    codes[rng.integers(0, out, (TERMS, n_in)), np.arange(n_in)] = rng.integers(1, 16, (TERMS, n_in))
    scales = np.empty((out, nb), dtype=np.uint8)
    for o in range(out):
        scales[o] = _near(kinds, rng)
    for run in range((nb + 7) // 8):
        group = (groups - 1, None, groups // 2, 0)[run % 4]
        if group is None:
            continue
        for b in rng.permutation(np.arange(8 * run, min(nb, 8 * run + 8)))[:3]:
            o = int(rng.integers(256 * group, min(out, 256 * group + 256)))
            kind = kinds[b]
            scales[o, b] = rng.integers(FAR[kind][0], FAR[kind][1] + 1)
            codes[o, 32 * b:32 * b + 32] = 0 if kind == USUAL else rng.integers(1, 16, 32)
    packed = MO.pack(codes)
    w = MO.dequant(packed, scales)
    assert (np.abs(w).sum(0) * 2047 < np.repeat(UNIT[kinds], 32) * 2.0 ** 24).all()
    assert ((w / np.repeat(UNIT[kinds], 32)) % 1 == 0).all()
    return packed, scales, w


# by the present rules: whole-row wavefronts; 16-row tiles; the tile kernel's shapes of 32, 64 and
# 128 tokens, each without and with K split over workgroups, each with more than eight groups of K
# for a share of them somewhere
PRODUCTS = [(1, 330, 2080), (2, 330, 2080), (1, 9001, 2080), (6, 330, 4640), (13, 330, 4640),
            (40, 1030, 4640), (100, 1030, 1184), (200, 4099, 9376), (77, 515, 27680),
            (300, 4099, 9376), (128, 2080, 4640), (1900, 3900, 5216), (700, 3001, 5216)]


@pytest.mark.parametrize("batch,out,n_in", PRODUCTS)
def test_products_where_float16_meets_far_scales_exact(batch, out, n_in):
    packed, scales, w = far_rows(out, n_in, batch + out)
    layer = MxLayer(dev(packed), dev(scales))
    for dtype in HALVES:
        x = _integers(batch, n_in, dtype, n_in + batch)
        want = x @ w.T
        for power in (0, -14):
            xd = rounded(np.ldexp(x, power), dtype).to(DEV)
            y, ok = guarded((batch, out), dtype)
            layer.gemm(xd, out=y)
            same(y, rounded(np.ldexp(want, power), dtype))
            ok()
            if batch <= 8:
                y, ok = guarded((batch, out), dtype)
                mx_gemv_batched([layer], [xd], [y])
                same(y, rounded(np.ldexp(want, power), dtype))
                ok()


# the gradient's tile shapes, each without and with K split over workgroups
GRADIENTS = [(64, 2050, 8288), (40, 2600, 1056), (300, 4099, 5216), (300, 2600, 1056),
             (520, 2085, 4640), (1300, 4400, 2080)]


@pytest.mark.parametrize("batch,out,n_in", GRADIENTS)
def test_gradients_where_float16_meets_far_scales_exact(batch, out, n_in):
    packed, scales, w = far_columns(out, n_in, batch + out)
    layer = MxLayer(dev(packed), dev(scales))
    for dtype in HALVES:
        dy = _integers(batch, out, dtype, n_in + batch)
        want = dy @ w
        for power in (0, -14):
            dx, ok = guarded((batch, n_in), dtype)
            layer.grad_input(rounded(np.ldexp(dy, power), dtype).to(DEV), out=dx)
            same(dx, rounded(np.ldexp(want, power), dtype))
            ok()


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


# --- both sides microscaled -----------------------------------------------------
# whole-row wavefronts, 16- and 32-token tiles (more than one of them along the tokens too), the
# tile kernel's three shapes without and with K split over workgroups
BOTH = [(1, 330, 2080), (2, 330, 2080), (4, 4100, 2080), (5, 50, 16480), (3, 330, 4640), (12, 330, 4640),
        (20, 515, 2080), (40, 4099, 2080), (70, 4099, 1056), (100, 1030, 1184), (200, 4099, 9376),
        (77, 515, 27680), (300, 4099, 5216), (1300, 4400, 2080), (700, 3001, 9376)]


@pytest.mark.parametrize("batch,out,n_in", BOTH)
def test_both_microscaled_with_opposite_scales_exact(batch, out, n_in):
    """Scales 2^d and 2^-d of the two sides, another d in every block from -127 to 127 (bytes 0 to
    254): each product of two values is a multiple of 1/4 up to 36, and the sums are exact."""
    rng = np.random.default_rng(batch + out)
    nb = n_in // 32
    d = rng.integers(-127, 128, nb)
    d[rng.integers(0, nb)] = 127
    d[rng.integers(0, nb)] = -127
    packed = rng.integers(0, 256, (out, n_in // 2), dtype=np.uint8)
    xp = rng.integers(0, 256, (batch, n_in // 2), dtype=np.uint8)
    scales = np.repeat((127 + d).astype(np.uint8)[None], out, 0)
    xs = np.repeat((127 - d).astype(np.uint8)[None], batch, 0)
    plain = np.full_like(scales, 127), np.full_like(xs, 127)
    want = MO.dequant(xp, plain[1]) @ MO.dequant(packed, plain[0]).T
    assert 36 * 4 * n_in < 1 << 24
    for dtype in HALVES:
        y, ok = guarded((batch, out), dtype)
        MxLayer(dev(packed), dev(scales)).gemm_mx(dev(xp), dev(xs), dtype, out=y)
        same(y, rounded(want, dtype))
        ok()
    # single NaN blocks, in the last group of K and at the array's very end: their rows alone
    xs[batch // 2, nb - 1 - min(3, nb - 1)] = 255
    xs[batch - 1, nb - 1] = 255
    scales[out // 3, nb // 2] = scales[out - 1, nb - 1] = 255
    want[[batch // 2, batch - 1]] = np.nan
    want[:, [out // 3, out - 1]] = np.nan
    for dtype in HALVES:
        same(MxLayer(dev(packed), dev(scales)).gemm_mx(dev(xp), dev(xs), dtype), rounded(want, dtype))


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch", [1, 2, 8, 256])
def test_both_microscaled_every_pair_of_scales(batch, dtype):
    """1.5 * 2^(a - 127) * 2^(b - 127) for every pair of bytes: the product itself, whatever its
    factors, down to float32's subnormals, infinite above its range, and NaN with byte 255."""
    codes = np.zeros((256, 32), dtype=np.uint8)
    codes[:, 17] = 2
    scales = np.arange(256, dtype=np.uint8)[:, None]
    layer = MxLayer(dev(MO.pack(codes)), dev(scales))
    codes[:, 17] = 3
    xp = dev(MO.pack(codes))
    a = scales.astype(np.int64) - 127
    want = np.ldexp(1.5, a + a.T)                          # [x's byte, W's byte]
    want[255], want[:, 255] = np.nan, np.nan
    got = torch.cat([layer.gemm_mx(xp[i:i + batch], dev(scales[i:i + batch]), dtype)
                     for i in range(0, 256, batch)])
    same(got, rounded(want, dtype))
