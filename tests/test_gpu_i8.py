"""The int8 operators on the GPU against the float64 oracle.

Codes and scales have to be equal to the oracle's, bit for bit. A product's sum is
exact in whole numbers and what follows is three float32 operations in a stated
order, so it too is compared bit for bit, whatever the codes: a lost, doubled or
misplaced term cannot pass. The gated block's products likewise; its activation has
the tolerance of its float32 operations. Gradients are compared exactly where the
data allow it (terms of few bits) and elsewhere within one half step of float16 for
each term and one float32 rounding (a whole step, should the matrix instructions
truncate) of each addition.
"""
import numpy as np
import pytest
import torch

from additive_codebook_matmul_amd import AqlmError, I8Gated, I8Layer, i8_dequant, i8_quantize
from oracle import i8_oracle as IO
from test_gpu_mx import ALL, DEV, HALVES, dev, guarded, rounded, same

pytestmark = pytest.mark.gpu

ACTS = list(IO.ACTIVATIONS)


def half(a32, dtype):
    """float32 values rounded once to dtype."""
    with np.errstate(over="ignore"):
        return torch.from_numpy(np.ascontiguousarray(a32, dtype=np.float32)).to(dtype)


def weights(out, n_in, seed, low=-127, high=127):
    rng = np.random.default_rng(seed)
    codes = rng.integers(low, high + 1, (out, n_in)).astype(np.int8)
    scales = np.exp2(rng.uniform(-14, -6, out)).astype(np.float32)
    return codes, scales


def layer_of(w):
    return I8Layer(dev(w[0]), dev(w[1]))


def activations(batch, n_in, dtype, seed):
    """Normal values, rows of very different magnitude, one of zeros."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((batch, n_in)) * np.exp2(rng.integers(-6, 4, (batch, 1)))
    if batch > 2:
        x[1] = 0
    return rounded(x, dtype)


# --- quantisation and expansion ----------------------------------------------
def _values(rows, cols, dtype, seed):
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 12, (rows, 1)))
    v[::2] = np.round(v[::2]) / 2                     # ties where the largest is 127 or its multiple
    v[::2, 0] = 127 * np.exp2(rng.integers(-3, 3, v[::2, 0].shape))
    if rows > 2:
        v[1] = 0
        v[2] = np.finfo(np.float16).smallest_subnormal * rng.integers(-3, 4, cols)
    return rounded(v, dtype)


def _check_quantize(x):
    want_c, want_s = IO.quantize(x.double().numpy())
    codes, ok_c = guarded(tuple(x.shape), torch.int8)
    scales, ok_s = guarded((x.shape[0],), torch.float32)
    i8_quantize(x.to(DEV), out=(codes, scales))
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert np.array_equal(scales.cpu().numpy(), want_s, equal_nan=True)
    ok_c()
    ok_s()


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (5, 1024), (9, 528), (7, 4112), (130, 176), (600, 2064),
                                       (2, 8208), (2, 28672), (3, 70000), (1, 131056), (2, 140000)])
def test_quantize_codes_and_scales(rows, cols, dtype):
    _check_quantize(_values(rows, cols, dtype, rows + cols))


@pytest.mark.parametrize("dtype", HALVES)
def test_quantize_every_half(dtype):
    """All 65536 bit patterns, each the largest of a row and each beside a larger value."""
    every = torch.from_numpy(np.arange(65536, dtype=np.uint16).view(np.int16)).view(dtype)
    alone = torch.zeros((65536, 16), dtype=dtype)
    alone[:, 3] = every
    alone[:, 5] = every / 3
    _check_quantize(alone)
    finite = every[torch.isfinite(every)]
    beside = finite[torch.randperm(finite.numel(), generator=torch.Generator().manual_seed(1))][:63488]
    _check_quantize(beside.view(-1, 64))


def test_quantize_float32_extremes():
    rng = np.random.default_rng(3)
    x = rng.integers(0, 1 << 32, (256, 64), dtype=np.uint64).astype(np.uint32).view(np.float32)
    x[~np.isfinite(x)] = 1.0
    x[:64] = np.float32(2.0 ** -149) * rng.integers(-300, 300, (64, 64))
    x[64:96] *= np.float32(2.0 ** -100)
    x[96, 5], x[97, 40], x[98, 0] = np.inf, -np.inf, np.nan
    x[99] = np.float32(3.4e38)
    x[100:130] = rng.standard_normal((30, 64)) * np.float32(2.0 ** -101)
    _check_quantize(torch.from_numpy(x))


def test_quantize_near_ties_of_float32():
    """Values one float32 step around each middle of two codes, for many row maxima."""
    rng = np.random.default_rng(5)
    top = (rng.random(400) + 0.5).astype(np.float32)
    middle = (np.arange(127) + 0.5)[None, :] * top[:, None].astype(np.float64) / 127
    m = middle.astype(np.float32)
    x = np.concatenate([m, np.nextafter(m, np.float32(9)), np.nextafter(m, np.float32(0)), top[:, None],
                        np.zeros((400, 2), np.float32)], axis=1)
    _check_quantize(torch.from_numpy(x[:, :384].copy()))


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 160), (256, 256), (129, 2064), (2, 28672)])
def test_dequant(rows, cols, dtype):
    rng = np.random.default_rng(rows)
    codes = rng.integers(-128, 128, (rows, cols)).astype(np.int8)
    scales = np.exp2(rng.uniform(-20, 8, rows)).astype(np.float32)
    if rows > 2:
        scales[:3] = [np.nan, np.inf, 1e-42]
    out, ok = guarded((rows, cols), dtype)
    i8_dequant(dev(codes), dev(scales), dtype, out=out)
    with np.errstate(invalid="ignore"):
        same(out, half(codes.astype(np.float32) * scales[:, None], dtype))
    ok()


# --- products, exact ----------------------------------------------------------
# (batch, out, in): one to many tokens, odd and ragged sizes, every tile's edge
SHAPES = [(1, 1, 16), (1, 17, 48), (1, 300, 112), (1, 64, 4096), (1, 33, 11008), (2, 40, 160), (2, 1030, 28672),
          (3, 129, 2080), (4, 511, 400), (5, 256, 1040), (6, 77, 8208), (8, 100, 4096), (9, 65, 512), (16, 48, 128),
          (17, 200, 1136), (31, 70, 32), (33, 130, 976), (64, 257, 2048), (77, 301, 1392), (128, 64, 4096),
          (129, 515, 272), (200, 96, 8192), (257, 260, 544), (300, 1000, 1024), (513, 768, 256), (1030, 259, 160)]
# whole grids of the larger tiles with ragged ends on every side, sums split over
# workgroups, batches on the border of the kernels for few rows
LARGE = [(1030, 3075, 4240), (700, 5000, 4176), (300, 4099, 4272), (64, 2050, 8304), (40, 11008, 528),
         (12, 4100, 8192), (24, 1376, 16400)]


def product(x, w, dtype):
    xc, xs = IO.quantize(x.double().numpy())
    return IO.value(IO.sums(xc, w[0]), w[1], xs)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", SHAPES + LARGE)
def test_forward_exact(batch, out, n_in, dtype):
    w = weights(out, n_in, batch + out)
    x = activations(batch, n_in, dtype, n_in + batch)
    want = half(product(x, w, dtype), dtype)
    layer = layer_of(w)
    y, ok = guarded((batch, out), dtype)
    layer.forward(x.to(DEV), out=y)
    same(y, want)
    ok()
    codes, scales = i8_quantize(x.to(DEV))
    y, ok = guarded((batch, out), dtype)
    layer.gemm_i8(codes, scales, dtype, out=y)
    same(y, want)
    ok()


@pytest.mark.parametrize("batch,out,n_in", [(1, 40, 131056), (3, 33, 131056), (20, 64, 131056), (150, 260, 131056)])
def test_sums_at_the_limit_of_32_bits(batch, out, n_in):
    """Codes of -128 on both sides at the most columns there may be: 2147221504 in a sum."""
    codes, x = np.full((out, n_in), -128, np.int8), np.full((batch, n_in), -128, np.int8)
    codes[1::2] = 127
    one = np.float32(2.0 ** -16)
    w, s = (codes, np.full(out, one)), np.full(batch, one)
    want = half(IO.value(IO.sums(x, codes), w[1], s), torch.bfloat16)
    same(layer_of(w).gemm_i8(dev(x), dev(s), torch.bfloat16), want)
    assert 128 * 128 * n_in < 1 << 31


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch", [1, 3, 8, 20, 70, 300])
def test_values_that_are_no_numbers(batch, dtype):
    """Tokens with NaN or infinity give rows of NaN, channels with such scales columns, nothing else changes."""
    out, n_in = 140, 272
    w = weights(out, n_in, 5)
    w[1][3], w[1][77] = np.nan, np.inf
    x = activations(batch, n_in, dtype, 9)
    x[batch - 1, 7] = float("inf")
    x[batch // 2, 100] = float("nan")
    xc, xs = IO.quantize(x.double().numpy())
    want = IO.value(IO.sums(xc, w[0]), w[1], xs)
    same(layer_of(w).forward(x.to(DEV)), half(want, dtype))
    assert np.isnan(want[batch - 1]).all() and np.isnan(want[:, 3]).all()


# --- gated blocks -------------------------------------------------------------
def gated_tolerance(g, u, a, dtype):
    """Of h = act(g) u: half a step of the type (or of its subnormals), and the float32
    operations: g's own three roundings and the exponent's move e^z by 4 |z| 2^-24 of
    itself where |z| <= 2 |g| + g^2 + |g|^3 / 10 bounds the exponent of each
    activation; 32 more roundings cover the rest. (v_exp_f32 gives 0 below 2^-126.)"""
    z = np.minimum(2 * np.abs(g) + g * g + np.abs(g) ** 3 / 10, 200)
    h = np.abs(a * u)
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -133
    return torch.finfo(dtype).eps / 2 * h * 1.01 + h * (4 * z + 32) * 2.0 ** -24 + tiny + np.abs(g * u) * 2.0 ** -125


def gated_case(batch, out, n_in, dtype, seed=0):
    gate, up = weights(out, n_in, batch + out + seed), weights(out, n_in, batch + n_in + seed + 1)
    for w in (gate, up):   # products of the size of 1
        w[1][:] *= np.float32(64 / np.sqrt(n_in))
    return gate, up, activations(batch, n_in, dtype, n_in + batch + seed)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", SHAPES + LARGE)
def test_gated(batch, out, n_in, dtype):
    act = ACTS[(batch + out) % 3]
    gate, up, x = gated_case(batch, out, n_in, dtype)
    block = I8Gated(layer_of(gate), layer_of(up), act)
    y, ok = guarded((batch, out), dtype)
    block.forward(x.to(DEV), out=y)
    ok()
    g, u = product(x, gate, dtype), product(x, up, dtype)
    a, _ = IO.act(g, act)
    ref = a * u.astype(np.float64)
    with np.errstate(over="ignore"):
        top = torch.finfo(dtype).max
        far = np.abs(y.cpu().double().numpy() - np.clip(ref, -top, top))
    inside = np.abs(ref) < top
    assert (far <= gated_tolerance(g.astype(np.float64), u, a, dtype))[inside].all()
    h, gs, us = block.forward_saving(x.to(DEV))
    assert torch.equal(h, y)
    assert np.array_equal(gs.cpu().numpy(), g) and np.array_equal(us.cpu().numpy(), u)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("batch", [1, 4, 30, 200])
def test_gated_over_the_range_of_the_gate(batch, act):
    """Gates from -1000 to 1000, zeros and infinities: one column each, the other layer all ones."""
    out, n_in = 200, 32
    codes = np.zeros((out, n_in), np.int8)
    codes[:, 0] = 127
    g_scale = np.concatenate([np.linspace(-1000, 1000, 61), np.linspace(-12, 12, 121),
                              [0, 1e-30, -1e-30, 1e30, -1e30, 3e38, -3e38, np.inf, -np.inf, np.nan],
                              np.zeros(8)]).astype(np.float32) / np.float32(127)
    gate = (codes, g_scale)
    up = (codes, np.full(out, np.float32(1 / 127)))
    x = torch.zeros((batch, n_in), dtype=torch.bfloat16)
    x[:, 0] = 1.0
    y = I8Gated(layer_of(gate), layer_of(up), act).forward(x.to(DEV)).cpu().double().numpy()
    g, u = product(x, gate, torch.bfloat16).astype(np.float64), product(x, up, torch.bfloat16).astype(np.float64)
    plain = np.isfinite(g)
    a, _ = IO.act(np.where(plain, g, 0), act)
    far = np.abs(y - a * u)
    assert (far <= gated_tolerance(np.clip(g, -1e6, 1e6), u, a, torch.bfloat16))[plain].all()
    assert np.isnan(y[np.isnan(g)]).all()
    assert np.isinf(y[g == np.inf]).all()


# --- gradients ----------------------------------------------------------------
def whole(rows, cols, seed, top=2):
    return np.random.default_rng(seed).integers(-top, top + 1, (rows, cols)).astype(np.float64)


def small_weights(out, n_in, seed):
    """Codes of few bits and powers of two: terms exact in float16, sums in float32."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(-3, 4, (out, n_in)).astype(np.int8)
    return codes, np.exp2(rng.integers(-3, 4, out)).astype(np.float32)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", SHAPES + LARGE)
def test_grad_input_exact(batch, out, n_in, dtype):
    w = small_weights(out, n_in, batch + out)
    dy = whole(batch, out, n_in + batch)
    ref, bound = IO.back(dy * w[1][None, :], w[0])
    assert bound.max() * 8 < 1 << 24               # multiples of 2^-3
    dx, ok = guarded((batch, n_in), dtype)
    layer_of(w).grad_input(rounded(dy, dtype).to(DEV), out=dx)
    same(dx, half(ref, dtype))
    ok()


def grad_tolerance(terms, ref, codes, dtype):
    """Half a step of the result, half a float16 step (11 significant bits: values of [1, 2) are
    2^-10 apart, so 2^-11 of the term) and three float32 roundings of each term (float16 below
    2^-14 of the token's 2^14: 2^-39 of the largest), and the additions'."""
    bound = np.abs(terms) @ np.abs(codes.astype(np.float64))
    top = np.abs(terms).max(axis=1, keepdims=True)
    flat = np.abs(codes.astype(np.float64)).sum(axis=0)[None, :] * top * 2.0 ** -39
    K = codes.shape[0]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134
    return (torch.finfo(dtype).eps / 2 * np.abs(ref) + bound * (2.0 ** -11 + 3 * 2.0 ** -24 + K * 2.0 ** -23)
            + flat + tiny)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", [(1, 40, 64), (5, 1000, 528), (77, 4099, 272), (300, 513, 1040),
                                            (600, 1376, 4096)])
def test_grad_input(batch, out, n_in, dtype):
    w = weights(out, n_in, out)
    rng = np.random.default_rng(batch)
    low = -6 if dtype == torch.float16 else -100     # rows of very different magnitude
    dy = rounded(rng.standard_normal((batch, out)) * np.exp2(rng.integers(low, 4, (batch, 1))), dtype)
    terms = dy.double().numpy() * w[1].astype(np.float64)[None, :]
    ref, _ = IO.back(terms, w[0])
    got = layer_of(w).grad_input(dy.to(DEV)).cpu().double().numpy()
    assert (np.abs(got - ref) <= grad_tolerance(terms, ref, w[0], dtype)).all()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", SHAPES + LARGE)
def test_gated_grad_exact(batch, out, n_in, dtype):
    """Gates of 64 and more, where act(g) = g and act'(g) = 1 in float32 too."""
    act = ACTS[(batch + n_in) % 3]
    gate, up = small_weights(out, n_in, batch + out), small_weights(out, n_in, batch + out + 1)
    rng = np.random.default_rng(batch)
    g, u = 64.0 * rng.integers(1, 3, (batch, out)), whole(batch, out, 3)
    dh = whole(batch, out, n_in + batch, 1)
    tg, tu = dh * u * gate[1][None, :], dh * g * up[1][None, :]
    (rg, bg), (ru, bu) = IO.back(tg, gate[0]), IO.back(tu, up[0])
    assert (bg + bu).max() * 8 < 1 << 30
    exact = (bg + bu).max() * 8 < 1 << 24
    dx, ok = guarded((batch, n_in), dtype)
    I8Gated(layer_of(gate), layer_of(up), act).grad_input(
        rounded(dh, dtype).to(DEV), dev(g.astype(np.float32)), dev(u.astype(np.float32)), out=dx)
    ok()
    if exact:
        same(dx, half(rg + ru, dtype))
    else:
        both, codes = np.concatenate([tg, tu], axis=1), np.concatenate([gate[0], up[0]])
        tol = grad_tolerance(both, rg + ru, codes, dtype)
        top = torch.finfo(dtype).max
        far = np.abs(dx.cpu().double().numpy() - np.clip(rg + ru, -top, top))
        assert (far <= tol)[np.abs(rg + ru) < top].all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", [(1, 40, 64), (6, 1000, 528), (77, 1377, 272), (260, 513, 1040)])
def test_gated_grad(batch, out, n_in, dtype, act):
    gate, up = weights(out, n_in, out), weights(out, n_in, out + 1)
    rng = np.random.default_rng(batch)
    g = (3 * rng.standard_normal((batch, out))).astype(np.float32)
    u = rng.standard_normal((batch, out)).astype(np.float32)
    g[0, :4] = [0, -30, 30, -90]
    dh = rounded(rng.standard_normal((batch, out)) * 0.02, dtype)
    tg, tu = IO.gated_terms(g.astype(np.float64), u.astype(np.float64), dh.double().numpy(),
                            gate[1].astype(np.float64), up[1].astype(np.float64), act)
    both, codes = np.concatenate([tg, tu], axis=1), np.concatenate([gate[0], up[0]])
    ref, bound = IO.back(both, codes)
    got = I8Gated(layer_of(gate), layer_of(up), act).grad_input(dh.to(DEV), dev(g), dev(u)).cpu().double().numpy()
    # and act' is a sum of two parts that may cancel (near g = -1.2): 64 float32
    # roundings of dh u (1 + g^2) w and dh g w each
    w64 = [w[1].astype(np.float64)[None, :] for w in (gate, up)]
    d64, g64 = np.abs(dh.double().numpy()), np.abs(g.astype(np.float64))
    slack = 64 * 2.0 ** -24 * (IO.back(d64 * np.abs(u) * (1 + g64 ** 2) * w64[0], np.abs(gate[0].astype(np.int16)))[0]
                               + IO.back(d64 * g64 * w64[1], np.abs(up[0].astype(np.int16)))[0])
    assert (np.abs(got - ref) <= grad_tolerance(both, ref, codes, dtype) + slack).all()


@pytest.mark.parametrize("dtype", HALVES)
def test_gradients_that_are_no_numbers(dtype):
    """Infinities and NaN of a token reach that token's gradient as the arithmetic has them, no other's."""
    out, n_in, batch = 70, 96, 5
    w = small_weights(out, n_in, 1)
    dy = whole(batch, out, 2)
    dy[1, 3], dy[2, 5], dy[3, 0], dy[3, 9] = np.inf, np.nan, np.inf, -np.inf
    dy[4] = 0
    with np.errstate(invalid="ignore"):
        ref = (dy * w[1][None, :]) @ w[0].astype(np.float64)
    same(layer_of(w).grad_input(rounded(dy, dtype).to(DEV)), half(ref, dtype))


@pytest.mark.parametrize("dtype", HALVES)
def test_refusals(dtype):
    w = weights(40, 64, 1)
    layer, x = layer_of(w), torch.zeros((2, 64), dtype=dtype, device=DEV)
    block = I8Gated(layer, layer)
    for bad in (x[:, :32], x.t(), x.float(), x.cpu(), x[0], torch.zeros((2, 80), dtype=dtype, device=DEV),
                torch.zeros((2, 128), dtype=dtype, device=DEV)[:, ::2]):
        with pytest.raises(ValueError):
            layer.forward(bad)
        with pytest.raises(ValueError):
            block.forward(bad)
        with pytest.raises(ValueError):
            block.forward_saving(bad)
    with pytest.raises(ValueError):
        layer.grad_input(x)
    with pytest.raises(ValueError):
        layer.forward(x, out=torch.empty((2, 41), dtype=dtype, device=DEV))
    with pytest.raises(ValueError):
        I8Gated(layer, layer_of(weights(41, 64, 1)))
    dh = torch.zeros((2, 40), dtype=dtype, device=DEV)
    g = torch.zeros((2, 40), device=DEV)
    for bad in (g.half(), g[:1], g.cpu(), torch.zeros((40, 2), device=DEV).t()):
        with pytest.raises(ValueError):
            block.grad_input(dh, g, bad)
        with pytest.raises(ValueError):
            block.grad_input(dh, bad, g)
    buf = torch.zeros(2 * 64 + 8, dtype=dtype, device=DEV)
    with pytest.raises(AqlmError):                    # off alignment
        layer.forward(buf[1:129].view(2, 64))
    with pytest.raises(ValueError):
        I8Layer(dev(w[0]), dev(w[1].astype(np.float64)))
    with pytest.raises(ValueError):
        I8Layer(dev(w[0])[:, :40], dev(w[1]))
    with pytest.raises(ValueError):
        I8Layer(dev(w[0]), dev(w[1])[:39])
    none = torch.zeros((0, 64), dtype=dtype, device=DEV)
    assert layer.forward(none).shape == (0, 40) and block.forward(none).shape == (0, 40)
    assert layer.grad_input(torch.zeros((0, 40), dtype=dtype, device=DEV)).shape == (0, 64)
    codes, scales = i8_quantize(none)
    assert codes.shape == (0, 64) and scales.shape == (0,) and i8_dequant(codes, scales).shape == (0, 64)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,cols", [(1, 128), (17, 16), (1000, 112), (4099, 128), (33, 144), (70001, 32)])
def test_conversion_of_short_rows(rows, cols, dtype):
    x = _values(rows, cols, dtype, rows)
    _check_quantize(x)
    codes, scales = IO.quantize(x.double().numpy())
    out, ok = guarded((rows, cols), dtype)
    i8_dequant(dev(codes), dev(scales), dtype, out=out)
    same(out, half(codes.astype(np.float32) * scales[:, None], dtype))
    ok()


@pytest.mark.parametrize("act", ACTS)
def test_gated_gradient_over_the_range_of_the_gate(act):
    """act' alone (up's scales are 0), a token for each gate, so that none hides below a larger one."""
    g1 = np.concatenate([np.linspace(-1000, 1000, 61), np.linspace(-12, 12, 121),
                         [0, 1e-30, -1e-30, 1e6, -1e6, 1e18, -1e18, 1e25, -1e25, 3e38, -3e38, np.nan]]).astype(np.float32)
    batch, out, n_in = len(g1), 8, 16
    codes = np.zeros((out, n_in), np.int8)
    codes[0, 0] = 1
    dh = torch.zeros((batch, out), dtype=torch.bfloat16)
    dh[:, 0] = 1.0
    g = np.zeros((batch, out), np.float32)
    g[:, 0] = g1
    gate, up = (codes, np.ones(out, np.float32)), (codes, np.zeros(out, np.float32))
    got = I8Gated(layer_of(gate), layer_of(up), act).grad_input(
        dh.to(DEV), dev(g), dev(np.ones((batch, out), np.float32))).cpu().double().numpy()
    plain = np.isfinite(g1)
    with np.errstate(over="ignore", under="ignore"):
        _, slope = IO.act(np.where(plain, g1.astype(np.float64), 0), act)
    # the roundings to float16 and bfloat16 are 2^-11 and 2^-8 at most; e^z is off by |z| 2^-23 of
    # itself and a few steps, with |z| at most 90 where it is not 0; act' is a sum of parts up to 1
    # + |g| that cancel near g = -1; from 2^-120 on down float32's e^z loses bits and vanishes
    near = np.clip(np.abs(np.where(plain, g1.astype(np.float64), 0)), 0, 14)
    tol = np.abs(slope) * (2.0 ** -11 + 2.0 ** -8 + 128 * 2.0 ** -23) + 16 * 2.0 ** -24 * np.exp2(-near) + 2.0 ** -120
    assert (np.abs(got[:, 0] - slope) <= tol)[plain].all()
    assert np.isnan(got[~plain, 0]).all()
    assert (got[:, 1:][plain] == 0).all()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", [(1, 40, 16384), (1, 37, 16400), (1, 21, 32768), (1, 20, 32784), (2, 37, 8192),
                                            (2, 37, 8208), (2, 20, 16384), (2, 21, 16400), (3, 20, 4112), (1, 21, 65536),
                                            (1, 21, 131056), (2, 20, 32784), (2, 21, 131056), (4, 20, 16400), (4, 21, 131056),
                                            (8, 21, 131056)])
def test_long_rows_of_few_tokens(batch, out, n_in, dtype):
    """Around the lengths up to which a product's own workgroups quantise the tokens, and to which LDS holds them."""
    w, up = weights(out, n_in, n_in), weights(out, n_in, n_in + 1)
    x = activations(batch, n_in, dtype, out)
    y, ok = guarded((batch, out), dtype)
    layer_of(w).forward(x.to(DEV), out=y)
    ok()
    same(y, half(product(x, w, dtype), dtype))
    h, g, u = I8Gated(layer_of(w), layer_of(up)).forward_saving(x.to(DEV))
    assert np.array_equal(g.cpu().numpy(), product(x, w, dtype))
    assert np.array_equal(u.cpu().numpy(), product(x, up, dtype))
