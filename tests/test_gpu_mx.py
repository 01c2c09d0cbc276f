"""The microscaled (MXFP4) operators on the GPU against the float64 oracle.

Where the data allow it the comparison is exact: with small whole activations
and scales near 1 every partial sum is a multiple of 2^-3 below 2^21, so
float32 accumulation is exact in any order, and the result has to be the exact
sum rounded once (to nearest even) to the output's type, bit for bit. A lost,
doubled or misplaced product cannot pass. Elsewhere the tolerance is that of the
arithmetic: half a step of the output's type, and one float32 rounding (a whole
step, should the matrix instructions truncate) of each of the K additions,
|y - ref| <= eps/2 |ref| + K 2^-23 sum |x w|.
"""
import numpy as np
import pytest
import torch

from additive_codebook_matmul_amd import (AqlmError, AqlmLayer, MxLayer, mx_dequant,
                                          mx_gemv_batched, mx_quantize, workloads as WL)
from oracle import mx_oracle as MO

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
HALVES = [torch.float16, torch.bfloat16]
ALL = HALVES + [torch.float32]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def rounded(a, dtype):
    """float64 values to dtype: exact in float32 first where the tests need one rounding."""
    with np.errstate(over="ignore"):
        if dtype == torch.float16:
            return torch.from_numpy(a.astype(np.float16))
        return torch.from_numpy(a.astype(np.float32)).to(dtype)


def same(got, want):
    """Equal values, NaN with NaN (zeros of either sign are equal)."""
    g, w = got.cpu().double().numpy(), want.double().numpy()
    bad = ~((g == w) | (np.isnan(g) & np.isnan(w)))
    assert g.shape == w.shape
    assert not bad.any(), (int(bad.sum()), bad.size, np.argwhere(bad)[:4].tolist(),
                           g[bad][:4].tolist(), w[bad][:4].tolist())


def near(got, ref, bound, K, dtype):
    g = got.cpu().double().numpy()
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + K * 2.0 ** -23 * bound + 2.0 ** -24
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), g[bad][:4], ref[bad][:4])


def guarded(shape, dtype):
    """A contiguous tensor inside a buffer of sevens, and a check that the rest still is."""
    n = int(np.prod(shape))
    pad = 256 // torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((n + 2 * pad,), 7, dtype=dtype, device=DEV)

    def check():
        assert bool((buf[:pad] == 7).all()) and bool((buf[pad + n:] == 7).all())
    return buf[pad:pad + n].view(shape), check


def whole_weights(out, n_in, seed, low=125, high=129):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (out, n_in), dtype=np.uint8)
    scales = rng.integers(low, high + 1, (out, n_in // 32)).astype(np.uint8)
    packed = MO.pack(codes)
    return packed, scales, MO.dequant(packed, scales)


def whole(rows, cols, seed, top=2):
    return np.random.default_rng(seed).integers(-top, top + 1, (rows, cols)).astype(np.float64)


# --- quantisation and expansion ----------------------------------------------
def _values(rows, cols, dtype, seed):
    """Every magnitude the type has, ties of the 4-bit grid, zeros of both signs."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 12, (rows, 1)))
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 4.0, 0.0, -0.0])
    pick = rng.random((rows, cols)) < 0.4
    v = np.where(pick, rng.choice(ties, (rows, cols)) * rng.choice([-1.0, 1.0], (rows, cols)), v)
    v[0, :32] = 0.0
    if rows > 2:
        v[1, :32] = np.finfo(np.float16).smallest_subnormal * rng.integers(-3, 4, 32)
        v[2, :32] = 60000.0 * rng.choice([-1.0, 1.0], 32)
    return rounded(v, dtype)


@pytest.mark.parametrize("rule", ["floor", "ceil"])
@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (5, 1024), (7, 4128), (130, 160)])
def test_quantize_codes_and_scales(rows, cols, dtype, rule):
    x = _values(rows, cols, dtype, rows + cols)
    want_c, want_s = MO.quantize(x.double().numpy(), rule)
    codes, ok_c = guarded((rows, cols // 2), torch.uint8)
    scales, ok_s = guarded((rows, cols // 32), torch.uint8)
    mx_quantize(x.to(DEV), rule, out=(codes, scales))
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    ok_c()
    ok_s()


@pytest.mark.parametrize("rule", ["floor", "ceil"])
@pytest.mark.parametrize("dtype", HALVES)
def test_quantize_every_half(dtype, rule):
    """All 65536 bit patterns, each the largest of a block and each beside a larger value."""
    bits = np.arange(65536, dtype=np.uint16).view(np.int16)
    every = torch.from_numpy(bits).view(dtype)
    alone = torch.zeros((2048, 32 * 32), dtype=dtype)
    alone[:, ::32] = every.view(2048, 32)
    beside = every.view(2048, 32).repeat(1, 2)
    beside[:, 32] = 48.0
    for x in (alone, beside):
        want_c, want_s = MO.quantize(x.double().numpy(), rule)
        codes, scales = mx_quantize(x.to(DEV), rule)
        assert np.array_equal(scales.cpu().numpy(), want_s)
        assert np.array_equal(codes.cpu().numpy(), want_c)


@pytest.mark.parametrize("rule", ["floor", "ceil"])
def test_quantize_float32_extremes(rule):
    rng = np.random.default_rng(3)
    x = rng.integers(0, 1 << 32, (256, 64), dtype=np.uint64).astype(np.uint32).view(np.float32)
    x[np.isnan(x)] = 1.0
    x[:64] = np.float32(2.0 ** -149) * rng.integers(-9, 9, (64, 64))
    x[64:96] *= np.float32(2.0 ** -100)
    x[96, 5], x[97, 40], x[98, 0] = np.inf, -np.inf, np.nan
    x[99] = np.float32(3.4e38)
    want_c, want_s = MO.quantize(x.astype(np.float64), rule)
    codes, scales = mx_quantize(dev(x), rule)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)


@pytest.mark.parametrize("dtype", ALL)
def test_dequant_every_code_and_scale(dtype):
    codes = np.tile(np.arange(32, dtype=np.uint8) % 16, (256, 1))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    packed = MO.pack(codes)
    out, ok = guarded((256, 32), dtype)
    mx_dequant(dev(packed), dev(scales), dtype, out=out)
    want = MO.dequant(packed, scales)
    same(out, rounded(want, dtype))
    zero = dev(packed)[:, :1] == 0x10
    assert bool(zero.all())
    assert bool(torch.signbit(out[127, 8]).item())      # code 8 is -0
    ok()


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 160), (129, 2080), (1000, 1024)])
def test_dequant_shapes(rows, cols, dtype):
    packed, scales, w = whole_weights(rows, cols, 5, 100, 150)
    out, ok = guarded((rows, cols), dtype)
    mx_dequant(dev(packed), dev(scales), dtype, out=out)
    same(out, rounded(w, dtype))
    ok()


# --- products, exact ----------------------------------------------------------
# (batch, out, in): one to many tokens, odd and ragged sizes, every tile's edge
SHAPES = [(1, 1, 32), (1, 17, 64), (1, 300, 96), (1, 64, 4096), (1, 33, 11008), (2, 40, 160),
          (3, 129, 2080), (5, 256, 1056), (8, 100, 4096), (9, 65, 512), (16, 48, 128),
          (17, 200, 1120), (31, 70, 32), (33, 130, 992), (64, 257, 2048), (77, 301, 1376),
          (128, 64, 4096), (129, 515, 288), (200, 96, 8192), (257, 260, 544), (300, 1000, 1024),
          (513, 768, 256), (1030, 259, 160)]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", SHAPES)
def test_gemm_exact(batch, out, n_in, dtype):
    packed, scales, w = whole_weights(out, n_in, batch + out)
    x = whole(batch, n_in, n_in + batch)
    y, ok = guarded((batch, out), dtype)
    layer = MxLayer(dev(packed), dev(scales))
    layer.gemm(rounded(x, dtype).to(DEV), out=y)
    want = rounded(MO.product(x, w)[0], dtype)
    same(y, want)
    ok()
    same(layer.forward(rounded(x, dtype).to(DEV)), want)
    if batch <= 8:
        same(layer.gemv(rounded(x, dtype).to(DEV)), want)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", SHAPES)
def test_gemm_mx_exact(batch, out, n_in, dtype):
    packed, scales, w = whole_weights(out, n_in, batch + out)
    xp, xs, x = whole_weights(batch, n_in, 7 * batch + n_in, 127, 128)
    y, ok = guarded((batch, out), dtype)
    MxLayer(dev(packed), dev(scales)).gemm_mx(dev(xp), dev(xs), dtype, out=y)
    # products reach 6 * 24 * 2 and are multiples of 2^-4: 2^-4 * 2^24 holds every sum
    assert n_in * 288 * 16 <= 1 << 24 or MO.product(x, w)[1].max() * 16 < 1 << 24
    same(y, rounded(MO.product(x, w)[0], dtype))
    ok()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", SHAPES + [(4, 11008, 64), (40, 4099, 96), (300, 2051, 320)])
def test_grad_input_exact(batch, out, n_in, dtype):
    packed, scales, w = whole_weights(out, n_in, batch + out)
    dy = whole(batch, out, n_in + batch)
    dx, ok = guarded((batch, n_in), dtype)
    MxLayer(dev(packed), dev(scales)).grad_input(rounded(dy, dtype).to(DEV), out=dx)
    same(dx, rounded(MO.grad_input(dy, w)[0], dtype))
    ok()


@pytest.mark.parametrize("rule", ["floor", "ceil"])
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", [(1, 40, 32), (2, 129, 2080), (9, 65, 4128), (77, 301, 1376), (300, 520, 1024)])
def test_forward_mx_gives_the_bits_of_its_parts(batch, out, n_in, dtype, rule):
    layer, _ = _layer(out, n_in, 2)
    x = rounded(np.random.default_rng(batch).standard_normal((batch, n_in)) * 3, dtype).to(DEV)
    y, ok = guarded((batch, out), dtype)
    layer.forward_mx(x, rule, out=y)
    ok()
    assert torch.equal(y, layer.gemm_mx(*mx_quantize(x, rule), dtype))


# Whole grids of the larger tiles with ragged ends on every side, more than 128
# blocks a row (scales staged again), rows whose blocks and scales end inside
# words and lines, K split over workgroups, and batches on the border of the
# kernels for few rows.
LARGE = [(1030, 3075, 4256), (700, 5000, 4192), (300, 4099, 4256), (64, 2050, 8288),
         (12, 9000, 4256), (16, 28672, 1056), (2, 28672, 4128), (8, 20011, 4160), (1500, 2104, 4384)]


@pytest.mark.parametrize("batch,out,n_in", LARGE)
def test_large_products_and_gradients_exact(batch, out, n_in):
    packed, scales, w = whole_weights(out, n_in, batch + out)
    xp, xs, xm = whole_weights(batch, n_in, 7 * batch + n_in, 127, 128)
    x, dy = whole(batch, n_in, n_in + batch), whole(batch, out, n_in + batch)
    assert (np.abs(xm) @ np.abs(w).T).max() * 16 < 1 << 24
    layer = MxLayer(dev(packed), dev(scales))
    want_y, want_mx, want_dx = x @ w.T, xm @ w.T, dy @ w
    for dtype in HALVES:
        y, ok_y = guarded((batch, out), dtype)
        same(layer.gemm(rounded(x, dtype).to(DEV), out=y), rounded(want_y, dtype))
        ok_y()
        y, ok_y = guarded((batch, out), dtype)
        same(layer.gemm_mx(dev(xp), dev(xs), dtype, out=y), rounded(want_mx, dtype))
        ok_y()
        dx, ok_dx = guarded((batch, n_in), dtype)
        same(layer.grad_input(rounded(dy, dtype).to(DEV), out=dx), rounded(want_dx, dtype))
        ok_dx()


# A few rows of activations, with rows of W longer than the part of x that a
# workgroup holds, ends inside every unit, and W on both sides of the choice of
# kernel.
FEW = [(1, 50, 65600), (1, 50, 16416), (1, 8200, 96), (2, 70, 8224), (2, 33, 20000), (2, 9001, 64),
       (3, 20, 20512), (4, 35, 16448), (5, 18, 12320), (6, 21, 10272), (5, 8193, 160),
       (6, 9000, 288), (7, 40, 12320), (8, 33, 16416)]


@pytest.mark.parametrize("batch,out,n_in", FEW)
def test_few_rows_exact(batch, out, n_in):
    packed, scales, w = whole_weights(out, n_in, batch + out)
    xp, xs, xm = whole_weights(batch, n_in, 7 * batch + n_in, 127, 128)
    x = whole(batch, n_in, n_in + batch)
    assert (np.abs(xm) @ np.abs(w).T).max() * 16 < 1 << 24
    layer = MxLayer(dev(packed), dev(scales))
    want_y, want_mx = x @ w.T, xm @ w.T
    for dtype in HALVES:
        xd = rounded(x, dtype).to(DEV)
        for call, want in ((lambda y: layer.gemm(xd, out=y), want_y),
                           (lambda y: mx_gemv_batched([layer], [xd], [y]), want_y),
                           (lambda y: layer.gemm_mx(dev(xp), dev(xs), dtype, out=y), want_mx),
                           (lambda y: layer.forward_mx(xd, "floor", out=y), want_y),
                           (lambda y: layer.forward_mx(xd, "ceil", out=y), want_y)):
            y, ok = guarded((batch, out), dtype)
            call(y)
            same(y, rounded(want, dtype))
            ok()


@pytest.mark.parametrize("rule", ["floor", "ceil"])
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch", [1, 2, 3, 4, 5, 6])
def test_quantised_on_the_way_like_by_itself(batch, dtype, rule):
    """Activations of every size, blocks of zeros, infinities and NaN: what the product quantises
    on the way is what mx_quantize gives (a block of 32 times one-hot rows of W, exactly)."""
    n_in = 32 * 70
    x = _values(batch, n_in, dtype, batch)
    if batch > 3:
        x[2, 2000], x[3, 100] = float("nan"), float("-inf")
    w = np.zeros((n_in, n_in), dtype=np.uint8)
    w[np.arange(n_in), np.arange(n_in)] = 2                    # 1.0
    layer = MxLayer(dev(MO.pack(w)), torch.full((n_in, n_in // 32), 127, dtype=torch.uint8, device=DEV))
    got = layer.forward_mx(x.to(DEV), rule)
    q = mx_dequant(*mx_quantize(x.to(DEV), rule), torch.float32).cpu().double()
    bad = q.isnan().view(batch, -1, 32).any(2)                 # NaN blocks reach every row of W
    rows = ~bad.any(1)
    want = q.float().to(dtype)
    assert torch.equal(got.cpu()[rows] + 0.0, want[rows] + 0.0)
    assert bool(got.cpu()[~rows].isnan().all())


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows", [4095, 8193, 32769])
def test_large_matrices_convert_like_their_parts(rows, dtype):
    """Matrices read and written past the caches (from 64 and 256 MiB on): every row's bits are
    those of the row's own small matrix."""
    cols = 4128
    gen = torch.Generator(device=DEV)
    gen.manual_seed(rows)
    x = torch.randn((rows, cols), generator=gen, device=DEV).to(dtype)
    for rule in ("floor", "ceil"):
        codes, scales = mx_quantize(x, rule)
        w = mx_dequant(codes, scales, dtype)
        for at in range(0, rows, 1000):
            part = mx_quantize(x[at:at + 1000].contiguous(), rule)
            assert torch.equal(codes[at:at + 1000], part[0])
            assert torch.equal(scales[at:at + 1000], part[1])
            assert torch.equal(w[at:at + 1000], mx_dequant(*part, dtype))


@pytest.mark.parametrize("dtype", HALVES)
def test_arrays_past_32_bit_offsets(dtype):
    """Codes, activations and results above 4 GiB: the far end's results are those of the far end
    alone. Whole numbers: exact whatever the kernels' order."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)

    def packed(rows, cols):
        codes = torch.randint(0, 256, (rows, cols // 2), generator=gen, device=DEV, dtype=torch.uint8)
        return codes, torch.full((rows, cols // 32), 127, device=DEV, dtype=torch.uint8)

    def halves(rows, cols):
        return torch.randint(-2, 3, (rows, cols), generator=gen, device=DEV, dtype=torch.int8).to(dtype)

    rows, cols, end = 600_000, 16384, 1000                # 4.9 GB of codes
    codes, scales = packed(rows, cols)
    layer = MxLayer(codes, scales)
    far = MxLayer(codes[-end:].clone(), scales[-end:].clone())
    for batch in (1, 3, 40):
        x = halves(batch, cols)
        assert torch.equal(layer.gemm(x)[:, -end:], far.gemm(x))
        mx = mx_quantize(x)
        assert torch.equal(layer.gemm_mx(*mx, dtype)[:, -end:], far.gemm_mx(*mx, dtype))
        dy = torch.zeros((batch, rows), dtype=dtype, device=DEV)
        dy[:, -end:] = halves(batch, end)
        assert torch.equal(layer.grad_input(dy), far.grad_input(dy[:, -end:].contiguous()))
    del codes, scales, layer, far, dy

    batch, cols = 1 << 20, 2080                           # 4.4 GB of activations and of results
    layer = MxLayer(*packed(2088, cols))
    x = halves(batch, cols)
    tail = x[-end:].clone()
    assert torch.equal(layer.gemm(x)[-end:], layer.gemm(tail))
    dy = halves(batch, 2088)
    assert torch.equal(layer.grad_input(dy)[-end:], layer.grad_input(dy[-end:].clone()))
    del dy
    mx = mx_quantize(x)
    small = mx_quantize(tail)
    assert torch.equal(mx[0][-end:], small[0]) and torch.equal(mx[1][-end:], small[1])
    assert torch.equal(layer.gemm_mx(*mx, dtype)[-end:], layer.gemm_mx(*small, dtype))
    assert torch.equal(mx_dequant(*mx, dtype)[-end:], tail)


# --- products, real data ------------------------------------------------------
REAL = [(1, 300, 4096), (4, 129, 11008), (16, 257, 1056), (50, 200, 4096), (130, 300, 2048),
        (300, 520, 1024)]


def _layer(out, n_in, seed, dtype=torch.float16):
    rng = np.random.default_rng(seed)
    W = rounded(rng.standard_normal((out, n_in)) * 0.02, dtype).to(DEV)
    layer = MxLayer.quantize(W)
    return layer, MO.dequant(layer.codes.cpu().numpy(), layer.scales.cpu().numpy())


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", REAL)
def test_products_of_real_data(batch, out, n_in, dtype):
    layer, w = _layer(out, n_in, batch)
    rng = np.random.default_rng(batch + 1)
    x = rounded(rng.standard_normal((batch, n_in)), dtype)
    dy = rounded(rng.standard_normal((batch, out)) * 0.01, dtype)
    xd = x.double().numpy()
    near(layer.forward(x.to(DEV)), *MO.product(xd, w), n_in, dtype)
    near(layer.grad_input(dy.to(DEV)), *MO.grad_input(dy.double().numpy(), w), out, dtype)
    q = MO.dequant(*MO.quantize(xd))
    near(layer.forward_mx(x.to(DEV)), *MO.product(q, w), n_in, dtype)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch", [1, 6, 20, 100, 300])
def test_scales_far_from_one(batch, dtype):
    """Scales that float16 cannot hold in the weights, next to ones that it can, with activations
    that use all eleven bits: the sums stay those of the exact weights."""
    out, n_in = 192, 512
    rng = np.random.default_rng(batch)
    codes = rng.integers(0, 16, (out, n_in), dtype=np.uint8)
    scales = np.full((out, n_in // 32), 120, dtype=np.uint8)
    scales[:64] = rng.integers(60, 104, (64, n_in // 32))       # below float16's subnormals
    scales[64:128] = rng.integers(98, 112, (64, n_in // 32))    # across the border
    scales[130] = 145                                           # products near 2^20
    scales[131] = 0
    packed = MO.pack(codes)
    w = MO.dequant(packed, scales)
    layer = MxLayer(dev(packed), dev(scales))
    x = rounded(rng.standard_normal((batch, n_in)) * 2.0 ** -12, dtype)
    big = rounded(rng.standard_normal((batch, n_in)) * 2.0 ** 13, dtype)
    for v in (x, big):
        ref, bound = MO.product(v.double().numpy(), w)
        got = layer.forward(v.to(DEV)).cpu().double().numpy()
        fits = np.abs(ref) < 60000
        tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + n_in * 2.0 ** -23 * bound
        tol += float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps
        assert (np.abs(got - ref) <= tol)[fits].all()
    dy = rounded(rng.standard_normal((batch, out)) * 2.0 ** -8, dtype)
    ref, bound = MO.grad_input(dy.double().numpy(), w)
    got = layer.grad_input(dy.to(DEV)).cpu().double().numpy()
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + out * 2.0 ** -23 * bound + 2.0 ** -24
    assert (np.abs(got - ref) <= tol)[np.abs(ref) < 60000].all()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch", [2, 8, 24, 100, 280])
def test_nan_and_infinity_propagate(batch, dtype):
    """A NaN scale spoils its output column (its input columns in the gradient), a NaN or infinite
    activation its row, and nothing else."""
    out, n_in = 200, 288
    packed, scales, w = whole_weights(out, n_in, batch)
    scales[130, 7] = 255
    w = MO.dequant(packed, scales)
    layer = MxLayer(dev(packed), dev(scales))
    x, dy = whole(batch, n_in, 1), whole(batch, out, 2)
    x[1, n_in - 1] = np.nan
    dy[1, out - 1] = np.nan
    with np.errstate(invalid="ignore"):
        same(layer.forward(rounded(x, dtype).to(DEV)), rounded(MO.product(x, w)[0], dtype))
        same(layer.grad_input(rounded(dy, dtype).to(DEV)), rounded(MO.grad_input(dy, w)[0], dtype))
        q = MO.dequant(*MO.quantize(x))
        same(layer.forward_mx(rounded(x, dtype).to(DEV)), rounded(MO.product(q, w)[0], dtype))
    x[1, n_in - 1] = np.inf
    codes = MO.unpack(packed)                            # inf * 0 is NaN: no zero codes
    codes[MO.E2M1[codes] == 0] = 1
    layer = MxLayer(dev(MO.pack(codes)), dev(scales))
    one = MO.dequant(MO.pack(codes), scales)
    same(layer.forward(rounded(x, dtype).to(DEV)), rounded(MO.product(x, one)[0], dtype))


# --- grouped calls, sequences, streams, graphs --------------------------------
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch", [1, 3, 8])
def test_grouped_layers(batch, dtype):
    """Up to 40 layers of different shapes in one call give the bits of single calls."""
    shapes = [(96, 2080), (1, 32), (333, 256), (16, 11008)] + [(17 + i, 64 + 32 * i) for i in range(36)]
    layers = [_layer(o, i, k)[0] for k, (o, i) in enumerate(shapes)]
    xs = [rounded(np.random.default_rng(k).standard_normal((batch, i)), dtype).to(DEV)
          for k, (o, i) in enumerate(shapes)]
    for n in (1, 2, 16, 17, 40):
        outs = [guarded((batch, o), dtype) for o, _ in shapes[:n]]
        mx_gemv_batched(layers[:n], xs[:n], [o for o, _ in outs])
        for k in range(n):
            assert torch.equal(outs[k][0], layers[k].gemv(xs[k]))
            outs[k][1]()
    shared = mx_gemv_batched([layers[0], layers[0]], [xs[0], xs[0]])
    assert torch.equal(shared[0], shared[1])


@pytest.mark.parametrize("batch", [1, 2, 8])
def test_grouped_layers_with_far_scales(batch):
    """The bits of single calls too where some rows have scales that float16 weights cannot take
    (their neighbours' sums must not depend on which rows a launch puts together)."""
    rng = np.random.default_rng(batch)
    layers, xs = [], []
    for k, (out, n_in) in enumerate([(1000, 2080), (1100, 2080), (16001, 1056), (20, 4128)]):
        w = MO.pack(rng.integers(0, 16, (out, n_in), dtype=np.uint8))
        scales = rng.integers(110, 125, (out, n_in // 32)).astype(np.uint8)
        far = rng.random(scales.shape) < 0.01
        scales[far] = rng.integers(85, 104, int(far.sum()))
        layers.append(MxLayer(dev(w), dev(scales)))
        xs.append(torch.from_numpy(rng.standard_normal((batch, n_in)).astype(np.float16)).to(DEV))
    alone = [layer.gemv(x) for layer, x in zip(layers, xs)]
    for n in (2, 3, 4):
        for got, want in zip(mx_gemv_batched(layers[:n], xs[:n]), alone):
            assert torch.equal(got, want)
    for layer, x, want in zip(layers, xs, alone):
        assert torch.equal(layer.gemm(x), want)


@pytest.mark.parametrize("batch", [1, 3, 8])
@pytest.mark.parametrize("out", [1, 20, 33, 64])
def test_grouped_layers_of_one_size(out, batch):
    """Query, key and value of one input, the results allocated by the call."""
    layers = [_layer(out, 96, k)[0] for k in range(3)]
    x = rounded(whole(batch, 96, 5), torch.float16).to(DEV)
    got = mx_gemv_batched(layers, [x, x, x])
    for y, layer in zip(got, layers):
        assert y.is_contiguous() and y.data_ptr() % 16 == 0
        assert torch.equal(y, layer.gemv(x))
    with pytest.raises(ValueError):
        mx_gemv_batched(layers, [x, x, x[:, :64]])
    with pytest.raises(ValueError):
        mx_gemv_batched(layers[:1], [torch.zeros((), dtype=torch.float16, device=DEV)])


def test_codebook_layer_to_microscaled_and_back():
    """A codebook layer's weights expanded, microscaled, and run as a step of adapter training: the
    forward products, and the gradient against differences of the forward (exact numbers)."""
    codes, books, scales, _ = WL.small_case(40, 64, WL.S2x8, 1, seed=1)
    dense = AqlmLayer(dev(codes), dev(books), dev(scales)).dequant()
    layer = MxLayer.quantize(dense)
    want_c, want_s = MO.quantize(dense.cpu().double().numpy())
    assert np.array_equal(layer.codes.cpu().numpy(), want_c)
    assert np.array_equal(layer.scales.cpu().numpy(), want_s)
    packed, s, w = whole_weights(40, 64, 9, 127, 127)
    for dtype in HALVES:
        layer = MxLayer(dev(packed), dev(s))
        x = whole(6, 64, 1, top=1)
        dy = whole(6, 40, 2, top=1)
        grad = layer.grad_input(rounded(dy, dtype).to(DEV)).cpu().double().numpy()
        assert dtype == torch.bfloat16 or np.array_equal(grad, dy @ w)
        near(layer.grad_input(rounded(dy, dtype).to(DEV)), *MO.grad_input(dy, w), 40, dtype)
        if dtype == torch.float16:      # sums are multiples of 0.5 below 1024: exact in float16
            for i in (0, 1, 31, 32, 63):
                up, down = x.copy(), x.copy()
                up[:, i] += 1
                down[:, i] -= 1
                y1 = layer.forward(rounded(up, dtype).to(DEV)).cpu().double().numpy()
                y0 = layer.forward(rounded(down, dtype).to(DEV)).cpu().double().numpy()
                assert np.array_equal(((y1 - y0) * dy).sum(1) / 2, grad[:, i])


def test_empty_batches():
    layer, _ = _layer(48, 96, 1)
    for dtype in HALVES:
        x = torch.empty((0, 96), dtype=dtype, device=DEV)
        assert layer.forward(x).shape == (0, 48) and layer.forward_mx(x).shape == (0, 48)
        assert layer.gemv(x).shape == (0, 48)
        assert layer.grad_input(torch.empty((0, 48), dtype=dtype, device=DEV)).shape == (0, 96)
    c, s = mx_quantize(torch.empty((0, 64), device=DEV))
    assert c.shape == (0, 32) and s.shape == (0, 2)
    assert mx_dequant(c, s).shape == (0, 64)


def test_refusals_on_the_device():
    layer, _ = _layer(48, 96, 1)
    x = torch.zeros((4, 96), dtype=torch.float16, device=DEV)
    bad = [lambda: layer.forward(x.float()), lambda: layer.forward(x[:, :64]),
           lambda: layer.forward(x.t()), lambda: layer.forward(x[:, ::2]), lambda: layer.forward(x[0]),
           lambda: layer.forward(x.cpu()), lambda: layer.grad_input(x),
           lambda: layer.gemm(x, out=torch.empty((4, 48), dtype=torch.bfloat16, device=DEV)),
           lambda: layer.gemm(x, out=torch.empty((48, 4), dtype=torch.float16, device=DEV).t()),
           lambda: layer.gemm_mx(*mx_quantize(x[:, :64].contiguous())),
           lambda: layer.gemm_mx(*mx_quantize(x), dtype=torch.float32),
           lambda: mx_quantize(x, rule="even"), lambda: mx_quantize(x.double()),
           lambda: mx_quantize(torch.zeros((4, 40), device=DEV)),
           lambda: mx_dequant(layer.codes, layer.scales, torch.float64),
           lambda: mx_dequant(layer.codes, layer.scales[:, :2].contiguous()),
           lambda: MxLayer(layer.codes.to(torch.int16), layer.scales),
           lambda: mx_gemv_batched([layer, layer], [x, x[:2].contiguous()]),
           lambda: mx_gemv_batched([layer, layer], [x, x.to(torch.bfloat16)]),
           lambda: mx_gemv_batched([layer], [x, x])]
    for k, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(k)
    with pytest.raises(AqlmError):                       # nine rows through the one-to-eight call
        layer.gemv(torch.zeros((9, 96), dtype=torch.float16, device=DEV))
    flat = torch.zeros(4 * 96 + 8, dtype=torch.float16, device=DEV)
    with pytest.raises(AqlmError):                       # two bytes off alignment
        layer.forward(flat[1:1 + 4 * 96].view(4, 96))


def _calls(dtype):
    layer, _ = _layer(520, 4096, 3)
    wide, _ = _layer(300, 1056, 4)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    x = {b: torch.randn((b, 4096), generator=gen, device=DEV).to(dtype) for b in (1, 5, 24, 100, 300)}
    dy = {b: torch.randn((b, 520), generator=gen, device=DEV).to(dtype) for b in (3, 70, 300)}
    xw = torch.randn((1, 1056), generator=gen, device=DEV).to(dtype)

    def run():
        got = []
        for b in x:
            got += [layer.forward(x[b]), layer.forward_mx(x[b])]
        for b in dy:
            got.append(layer.grad_input(dy[b]))
        got += mx_gemv_batched([layer, wide, layer], [x[1], xw, x[1]])
        codes, scales = mx_quantize(x[300], "ceil")
        return got + [codes, scales, mx_dequant(codes, scales, dtype)]
    return run


@pytest.mark.parametrize("dtype", HALVES)
def test_repeated_and_side_stream_calls_give_the_same_bits(dtype):
    run = _calls(dtype)
    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run()
    third = run()                        # on the default stream while the side stream works
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("dtype", HALVES)
def test_graph_replays_match_eager(dtype):
    run = _calls(dtype)
    eager = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run()
    for _ in range(4):
        for t in outs:
            t.fill_(1)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a, b)
        for a, b in zip(run(), eager):   # eager work between the replays
            assert torch.equal(a, b)
    del g
    torch.cuda.empty_cache()
