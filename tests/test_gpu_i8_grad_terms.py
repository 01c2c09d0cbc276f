"""The terms of int8 gradients: what enters the matrix instructions has float32's bits, not float16's.

A term (the incoming gradient times act' and the channel's scale) is handed on as two float16 numbers
that together hold 22 bits and more. Whole numbers of up to 16 bits therefore pass exactly, and where
their sums stay below 2^24 so does the whole gradient: compared bit for bit. Elsewhere the tolerance counts
the header's 2^-23 of a term (2^-50 of the token's largest) and float32's own roundings.
"""
import numpy as np
import pytest
import torch

from additive_codebook_matmul_amd import I8Gated, I8Layer
from oracle import i8_oracle as IO
from test_gpu_i8 import ACTS, half, layer_of, weights
from test_gpu_mx import DEV, HALVES, dev, guarded, rounded, same

pytestmark = pytest.mark.gpu

SIZES = [(1, 40, 64), (5, 1000, 528), (77, 4099, 272), (300, 513, 1040), (33, 8100, 96)]


def term_bits(K):
    """Bits of whole terms whose sums over K rows, two thirds of their codes not 0 and half of their
    gradients, stay below 2^24."""
    return min(16, 25 - int(np.ceil(np.log2(K + 1))))


def odd_scales(out, bits, seed):
    """Odd whole numbers of `bits` bits, times 2^-16: a gradient of them is below 2^8."""
    w = np.random.default_rng(seed).integers(1 << (bits - 1), 1 << bits, out) | 1
    return (w * 2.0 ** -16).astype(np.float32)


def signs(rows, cols, seed, zeros):
    """-1, 0 and 1."""
    rng = np.random.default_rng(seed)
    return (rng.integers(0, 2, (rows, cols)) * 2 - 1) * (rng.random((rows, cols)) >= zeros)


def layer_case(batch, out, n_in, dtype):
    """(weights, dy, gradient) of a layer, exact in float32."""
    w = signs(out, n_in, 1, 1 / 3).astype(np.int8), odd_scales(out, term_bits(out), out)
    dy = signs(batch, out, 2, 0.5)
    ref, bound = IO.back(dy * w[1].astype(np.float64)[None, :], w[0])
    assert bound.max() < 1 << 8
    return w, rounded(dy, dtype), ref


def gated_case(batch, out, n_in, dtype):
    """The same of a gated block, (gate, up, g, u, dh, gradient): gates of 64, where act(g) = g and act'(g) = 1
    in float32 too."""
    bits = term_bits(2 * out)
    gate = signs(out, n_in, 1, 1 / 3).astype(np.int8), odd_scales(out, bits, out)
    up = signs(out, n_in, 2, 1 / 3).astype(np.int8), odd_scales(out, bits, out + 1) / np.float32(64)
    dh, u = signs(batch, out, 3, 0.5), signs(batch, out, 4, 0)
    g = np.full((batch, out), 64.0)
    (rg, bg), (ru, bu) = (IO.back(dh * u * gate[1].astype(np.float64)[None, :], gate[0]),
                          IO.back(dh * g * up[1].astype(np.float64)[None, :], up[0]))
    assert (bg + bu).max() < 1 << 8
    return gate, up, dev(g.astype(np.float32)), dev(u.astype(np.float32)), rounded(dh, dtype), rg + ru


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", SIZES)
def test_whole_terms_of_a_layer(batch, out, n_in, dtype):
    w, dy, ref = layer_case(batch, out, n_in, dtype)
    dx, ok = guarded((batch, n_in), dtype)
    layer_of(w).grad_input(dy.to(DEV), out=dx)
    same(dx, half(ref, dtype))
    ok()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", SIZES)
def test_whole_terms_of_a_gated_block(batch, out, n_in, dtype):
    gate, up, g, u, dh, ref = gated_case(batch, out, n_in, dtype)
    dx, ok = guarded((batch, n_in), dtype)
    I8Gated(layer_of(gate), layer_of(up), ACTS[batch % 3]).grad_input(dh.to(DEV), g, u, out=dx)
    same(dx, half(ref, dtype))
    ok()


def tolerance(terms, ref, codes, dtype):
    """Half a step of the result's type; of each term 2^-23 (2^-50 of the token's largest) and one float32
    rounding, its scale's product; and a whole float32 step (should the matrix instructions truncate) of each
    of the 2 K additions, whose partial sums are at most the sum of magnitudes."""
    c = np.abs(codes.astype(np.float64))
    bound, K = np.abs(terms) @ c, codes.shape[0]
    flat = c.sum(axis=0)[None, :] * np.abs(terms).max(axis=1, keepdims=True) * 2.0 ** -50
    off = bound * (2.0 ** -23 + 2.0 ** -24 + 2 * K * 2.0 ** -23) * (1 + 2.0 ** -10) + flat
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134
    return torch.finfo(dtype).eps / 2 * (np.abs(ref) + off) + off + tiny


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", [(1, 1, 64), (7, 2, 256), (40, 24, 528), (300, 40, 272)])
def test_few_terms(batch, out, n_in, dtype):
    """Sums short enough that a term's bits show beside the additions'."""
    w = weights(out, n_in, out)
    dy = rounded(np.random.default_rng(batch).standard_normal((batch, out)), dtype)
    terms = dy.double().numpy() * w[1].astype(np.float64)[None, :]
    ref, _ = IO.back(terms, w[0])
    got = layer_of(w).grad_input(dy.to(DEV)).cpu().double().numpy()
    assert (np.abs(got - ref) <= tolerance(terms, ref, w[0], dtype)).all()


@pytest.mark.parametrize("batch", [1, 40, 300])
def test_terms_far_below_the_largest(batch):
    """The channel of a token's largest term has codes of 0 in every column but the first, so that terms down
    to 2^-40 of it are all that there is: each column has a term of its own."""
    out = n_in = 48
    rng = np.random.default_rng(3)
    codes = np.diag(rng.integers(64, 128, out)).astype(np.int8)
    codes[0, 0] = 1
    w = (codes, (np.exp2(-np.minimum(np.arange(out), 40)) * (1 + rng.random(out))).astype(np.float32))
    w[1][0] = 2.0
    dy = rounded(1 + rng.random((batch, out)), torch.bfloat16)
    terms = dy.double().numpy() * w[1].astype(np.float64)[None, :]
    ref, _ = IO.back(terms, codes)
    got = layer_of(w).grad_input(dy.to(DEV)).cpu().double().numpy()
    off = np.abs(ref) * (2.0 ** -23 + 2.0 ** -24 + 2.0 ** -22) + 128 * np.abs(terms).max(axis=1, keepdims=True) * 2.0 ** -50
    assert (np.abs(got - ref) <= (np.abs(ref) + off) * 2.0 ** -8 + off).all()


@pytest.mark.parametrize("batch,n_in", [(3, 16), (140, 16), (250, 4096)])
def test_the_most_rows_of_a_gated_block(batch, n_in):
    """With 4096 columns the tile is of 128 tokens, whose terms are 2^31 bytes. One 1 in each token's gradient (and
    a 2 in its last place): a result is a sum of four codes, exactly."""
    out = 1 << 21
    gen = torch.Generator(device="cuda")
    gen.manual_seed(batch)
    gate, up = (torch.randint(-127, 128, (out, n_in), generator=gen, device=DEV, dtype=torch.int8) for _ in range(2))
    dh = torch.zeros((batch, out), dtype=torch.float16, device=DEV)
    at = torch.randint(0, out - 1, (batch,), generator=gen, device=DEV)
    dh.scatter_(1, at[:, None], 1.0)
    dh[:, out - 1] = 2.0
    g, u = torch.full((batch, out), 64.0, device=DEV), torch.full((batch, out), 3.0, device=DEV)
    one = torch.ones(out, device=DEV)
    dx = I8Gated(I8Layer(gate, one), I8Layer(up, one / 64), "silu").grad_input(dh, g, u)
    want = 3 * (gate[at].float() + 2 * gate[out - 1].float()) + up[at].float() + 2 * up[out - 1].float()
    assert torch.equal(dx, want.half())
    del gate, up, dh, g, u, dx
    torch.cuda.empty_cache()
