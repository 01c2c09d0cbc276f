"""Every kernel that an int8 product or gradient can be done with, bit for bit.

Which tile a call takes is a modelled choice (csrc/i8_plan.hpp), so the sizes here are chosen by what they
reach: each tile shape, plain and gated, with K split over workgroups and not, with one and with several tiles
of tokens, rows a multiple of 8 and not, each remainder of the loop over the stages, ragged at every end.
test_i8_plans.py asks the choice itself and fails where a list leaves something out. References are products in
float64 (exact: sums stay below 2^53, a gradient's below 2^24) and the float32 operations of the header.
"""
import pytest
import torch

from additive_codebook_matmul_amd import I8Gated, I8Layer, i8_quantize
from test_gpu_mx import DEV, HALVES, guarded

pytestmark = pytest.mark.gpu

# (batch, out, in)
PRODUCTS = [
    (1, 1, 16), (5, 1, 16), (1, 8, 16), (22, 1, 16), (34, 1, 16), (5, 8, 16), (22, 8, 16), (33, 8, 16),
    (3, 1, 4560), (5, 1, 12992), (3, 8, 4112), (6, 8, 6192), (33, 1, 14960), (33, 8, 2112), (70, 10968, 16),
    (67, 35423, 16), (257, 13232, 16), (4458, 781, 16), (197, 34504, 16), (218, 37396, 16), (5, 38456, 720),
    (403, 22348, 16), (585, 16920, 16), (6, 37355, 784), (5, 31701, 1504), (6, 5080, 11936), (7, 6501, 8384),
    (71, 34533, 160), (5, 31464, 2512), (33, 17248, 704), (196, 16515, 144), (203, 16656, 144), (98, 8624, 656),
    (38, 16178, 1072), (260, 3867, 672), (2019, 71, 4784), (36, 16256, 1232), (38, 5232, 4144), (33, 16718, 1856),
    (70, 19327, 912), (2157, 72, 10400), (37, 4260, 11536), (40, 6344, 7200), (3947, 70, 6800), (372, 1000, 5264),
    (84, 36000, 656), (103, 2807, 6864), (141, 35248, 400), (33, 5516, 12048), (33, 8904, 7904), (159, 33400, 576),
    (193, 39834, 400), (3302, 138, 8800), (70, 11015, 5216), (202, 38172, 528), (2703, 400, 4496),
    (70, 12072, 5920), (148, 10952, 5616), (136, 7726, 9888), (3656, 536, 10000), (3751, 543, 10032),
    (3267, 1032, 8928), (203, 16392, 9776), (411, 5948, 14656), (216, 17735, 10384),
]
GATED = [
    (1, 1, 16), (5, 1, 16), (1, 8, 16), (9, 1, 16), (22, 1, 16), (5, 8, 16), (9, 8, 16), (22, 8, 16), (33, 8, 16),
    (36, 1, 2384), (67, 1, 1392), (9, 1, 15056), (11, 8, 4176), (35, 8, 2096), (68, 6320, 16), (67, 16776, 16),
    (195, 8336, 16), (3382, 534, 16), (199, 16807, 16), (205, 16656, 16), (5, 16741, 816), (405, 11242, 16),
    (5, 20112, 752), (419, 12464, 16), (5, 16048, 1600), (5, 5208, 6672), (6, 16274, 1936), (40, 8732, 656),
    (5, 5411, 8896), (2449, 771, 144), (3526, 133, 656), (1331, 37, 6480), (2181, 232, 656), (36, 1152, 8816),
    (36, 7872, 1472), (37, 7837, 1760), (36, 8616, 1872), (72, 8884, 992), (2108, 36, 10176), (33, 2072, 11712),
    (1434, 99, 6128), (66, 19688, 672), (33, 2766, 10288), (2794, 40, 8544), (34, 2157, 13264), (151, 16553, 400),
    (68, 17196, 880), (98, 1728, 6192), (130, 16824, 528), (35, 2912, 11600), (133, 11616, 944), (206, 17728, 400),
    (199, 17955, 544), (69, 5712, 4976), (3314, 72, 8336), (69, 6010, 5280), (2810, 202, 4512), (153, 3627, 8256),
    (139, 5528, 6368), (3739, 288, 10096), (3609, 270, 14096), (413, 2720, 13728), (198, 8400, 9456),
    (4274, 395, 9776), (207, 8241, 13200),
]
GRADS = [
    (1, 8, 16), (1, 1, 272), (1, 65, 16), (66, 1, 16), (1, 66, 144), (68, 1, 272), (33, 77, 16), (1, 6493, 16),
    (35, 657, 16), (33, 80, 144), (1, 10736, 144), (34, 584, 144), (1, 5208, 6832), (1661, 2636, 16),
    (4126, 216, 144), (33, 1904, 5584), (1355, 2132, 144), (41, 2568, 5424), (262, 2582, 1168), (2914, 401, 1296),
    (4236, 25464, 16), (65, 3272, 10912), (3001, 2864, 272),
]
GATED_GRADS = [
    (1, 1, 16), (1, 1, 144), (33, 1, 16), (33, 1, 144), (1, 3224, 16), (4200, 1, 144), (67, 1, 11280),
    (1, 4528, 176), (34, 272, 160), (34, 17880, 16), (1, 1384, 10912), (2732, 956, 16), (4662, 76, 144),
    (36, 1288, 3376), (45, 1064, 5408), (1395, 1050, 208), (108, 1296, 3120), (4435, 11376, 16), (3267, 272, 1104),
    (2766, 1528, 304), (77, 1504, 11152),
]
# and the sizes of Llama-2 layers
PRODUCTS += [(77, 4096, 11008), (1999, 4096, 11008), (16, 4096, 4096), (1, 8192, 28672)]
GATED += [(1, 11008, 4096), (8, 11008, 4096), (19, 28672, 8192), (2048, 11008, 4096), (333, 1376, 4096)]
GRADS += [(301, 4096, 11008), (2048, 11008, 4096)]
GATED_GRADS += [(333, 1376, 4096), (2048, 11008, 4096)]
# and one tile of tokens for the chip with K whole: many columns
GRADS += [(91, 968, 39152), (60, 689, 71376), (30, 1037, 37120), (21, 845, 30976)]
GATED_GRADS += [(113, 282, 98032), (56, 202, 68592), (3, 344, 68656), (24, 1189, 25264)]


def _gen(*sizes):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(hash(sizes) % (1 << 31))
    return gen


def _codes(rows, cols, gen, top=127):
    return torch.randint(-top, top + 1, (rows, cols), generator=gen, device=DEV, dtype=torch.int8)


def _scales(rows, gen):
    return torch.exp2(torch.rand(rows, generator=gen, device=DEV) * 4 - 16)


def _value(xc, xs, w):
    """float32 products: the exact sum, times the channel's scale, times the token's."""
    return ((xc.double() @ w[0].double().t()).float() * w[1]) * xs[:, None]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", PRODUCTS)
def test_product(batch, out, n_in, dtype):
    gen = _gen(batch, out, n_in)
    w = _codes(out, n_in, gen), _scales(out, gen)
    xc, xs = _codes(batch, n_in, gen), _scales(batch, gen) * 64
    xc[:, 0] = 127
    want = _value(xc, xs, w).to(dtype)
    layer = I8Layer(*w)
    y, ok = guarded((batch, out), dtype)
    layer.gemm_i8(xc, xs, dtype, out=y)
    assert torch.equal(y, want)
    ok()
    # and with x quantised in the call: whole numbers that reach 127 are their own codes, with scale 1
    want = _value(xc, torch.ones_like(xs), w).to(dtype)
    y, ok = guarded((batch, out), dtype)
    layer.forward(xc.to(dtype), out=y)
    assert torch.equal(y, want)
    ok()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", GATED)
def test_gated(batch, out, n_in, dtype):
    """g and u exactly. Gates from 32 on have silu(g) = g in float32, so that there h is g u rounded once."""
    gen = _gen(batch, out, n_in, 1)
    gate, up = ((_codes(out, n_in, gen), _scales(out, gen)) for _ in range(2))
    gate[1].mul_(2.0 ** 8)                        # (few gates of longer rows are between -128 and 32)
    up[1].mul_(2.0 ** -6)
    xc = _codes(batch, n_in, gen)
    xc[:, 0] = 127
    one = torch.ones(batch, device=DEV)
    g0, u0 = _value(xc, one, gate), _value(xc, one, up)
    block = I8Gated(I8Layer(*gate), I8Layer(*up), "silu")
    h, g, u = block.forward_saving(xc.to(dtype))
    assert torch.equal(g, g0) and torch.equal(u, u0)
    far = g0 >= 32
    assert torch.equal(h[far], (g0 * u0).to(dtype)[far])
    low = g0 <= -128                              # e^-128 is 0 in float32: h is 0
    assert bool((h[low] == 0).all()) and (batch * out < 64 or bool((far | low).any()))
    y, ok = guarded((batch, out), dtype)
    block.forward(xc.to(dtype), out=y)
    assert torch.equal(y, h)
    ok()


def _whole_terms(batch, out, K, gen):
    """-1, 0 and 1 as gradients, and odd scales of 12 bits (times 2^-16), so that the sum over K terms of that size
    and codes up to 7 stays below 2^24 times 2^-16: about 600 gradients of a token are not 0."""
    keep = torch.rand((batch, out), generator=gen, device=DEV) < min(0.5, 600 / K)
    sign = torch.randint(0, 2, (batch, out), generator=gen, device=DEV) * 2 - 1
    scales = [(torch.randint(1 << 11, 1 << 12, (out,), generator=gen, device=DEV) | 1) * 2.0 ** -16 for _ in range(2)]
    return torch.where(keep, sign, 0), scales


def _sum(terms, codes):
    bound = (terms.abs().double() @ codes.abs().double()).max()
    return terms.double() @ codes.double(), bound


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", GRADS)
def test_gradient(batch, out, n_in, dtype):
    gen = _gen(batch, out, n_in, 2)
    codes = _codes(out, n_in, gen, 7)
    dy, (scales, _) = _whole_terms(batch, out, out, gen)
    want, bound = _sum(dy.double() * scales.double(), codes)
    assert bound < 1 << 8
    dx, ok = guarded((batch, n_in), dtype)
    I8Layer(codes, scales).grad_input(dy.to(dtype), out=dx)
    assert torch.equal(dx, want.float().to(dtype))
    ok()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", GATED_GRADS)
def test_gated_gradient(batch, out, n_in, dtype):
    """Gates of 64, where silu(g) = g and its derivative is 1 in float32."""
    gen = _gen(batch, out, n_in, 3)
    gate, up = _codes(out, n_in, gen, 7), _codes(out, n_in, gen, 7)
    dh, (sg, su) = _whole_terms(batch, out, 2 * out, gen)
    su = su / 64
    g = torch.full((batch, out), 64.0, device=DEV)
    u = (torch.randint(0, 2, (batch, out), generator=gen, device=DEV) * 2 - 1).float()
    (a, ba), (b, bb) = _sum(dh.double() * u * sg.double(), gate), _sum(dh.double() * 64 * su.double(), up)
    assert ba + bb < 1 << 8
    dx, ok = guarded((batch, n_in), dtype)
    I8Gated(I8Layer(gate, sg), I8Layer(up, su), "silu").grad_input(dh.to(dtype), g, u, out=dx)
    assert torch.equal(dx, (a + b).float().to(dtype))
    ok()


def test_whole_numbers_are_their_own_codes():
    """What the tests above take from the quantisation."""
    gen = _gen(1)
    x = _codes(40, 272, gen)
    x[:, 0] = 127
    for dtype in HALVES:
        codes, scales = i8_quantize(x.to(dtype))
        assert torch.equal(codes, x) and bool((scales == 1).all())
