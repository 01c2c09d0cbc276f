"""int8 operators at their largest rows, columns and batch, where offsets pass 32 bits, checked on a
sample of results against whole-number sums."""
import numpy as np
import pytest
import torch

from additive_codebook_matmul_amd import I8Gated, I8Layer, i8_dequant, i8_quantize
from test_gpu_i8 import half
from test_gpu_mx import DEV, same

pytestmark = pytest.mark.gpu


def _codes(rows, cols, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randint(-127, 128, (rows, cols), generator=gen, device="cuda", dtype=torch.int8)


def _scales(rows, seed):
    return torch.from_numpy(np.exp2(np.random.default_rng(seed).integers(-16, -8, rows)).astype(np.float32)).to(DEV)


def _sample(n, count, seed):
    pick = np.random.default_rng(seed).choice(n, min(n, count), replace=False)
    return torch.from_numpy(np.unique(np.concatenate([[0, n - 1, n // 2], pick]))).to(DEV)


def _check_product(y, xc, xs, wc, ws, dtype):
    t, r = _sample(y.shape[0], 40, 1), _sample(y.shape[1], 200, 2)
    sums = xc[t].cpu().numpy().astype(np.float64) @ wc[r].cpu().numpy().astype(np.float64).T
    want = (sums.astype(np.float32) * ws[r].cpu().numpy()[None, :]) * xs[t].cpu().numpy()[:, None]
    same(y[t][:, r], half(want, dtype))


# (batch, out, in): results, weights and activations of more than 2^31 elements or bytes, the largest of each size
LARGE = [(300000, 8200, 32), (1 << 21, 64, 16), (3, 1 << 21, 16), (1500, 1 << 21, 48), (1, 40000, 65536),
         (20, 20000, 131056), (70, 20000, 131056), (20000, 300, 131056)]


@pytest.mark.parametrize("batch,out,n_in", LARGE)
def test_products(batch, out, n_in):
    wc, ws, xc, xs = _codes(out, n_in, 1), _scales(out, 1), _codes(batch, n_in, 2), _scales(batch, 2)
    y = I8Layer(wc, ws).gemm_i8(xc, xs, torch.bfloat16)
    _check_product(y, xc, xs, wc, ws, torch.bfloat16)


@pytest.mark.parametrize("batch,out,n_in", [(300000, 4100, 32), (1 << 21, 40, 16), (5, 1 << 20, 16), (40, 20000, 65536)])
def test_gated_products(batch, out, n_in):
    """The float32 products of both layers, and h where the gate is far from zero (gelu(g) = g)."""
    wc, uc = _codes(out, n_in, 1), _codes(out, n_in, 3)
    ws, us = torch.full((out,), 1.0, device=DEV), _scales(out, 4)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    x = torch.randn((batch, n_in), generator=gen, device="cuda", dtype=torch.bfloat16) * 20
    h, g, u = I8Gated(I8Layer(wc, ws), I8Layer(uc, us), "gelu").forward_saving(x)
    xc, xs = i8_quantize(x)
    _check_product(g, xc, xs, wc, ws, torch.float32)
    _check_product(u, xc, xs, uc, us, torch.float32)
    t, r = _sample(batch, 40, 1), _sample(out, 200, 2)
    gs, us_, hs = g[t][:, r].cpu(), u[t][:, r].cpu(), h[t][:, r].cpu()
    far = gs > 20
    assert bool(far.any())
    assert torch.equal((gs * us_).to(torch.bfloat16)[far], hs[far])


@pytest.mark.parametrize("batch,out,n_in", [(300000, 32, 8208), (1 << 21, 40, 48), (3, 1 << 21, 16), (600, 1 << 21, 32),
                                            (20, 20000, 131056), (20000, 300, 131056), (9000, 250000, 16)])
def test_input_gradients(batch, out, n_in):
    """dy of one 1 in each row (and a 2 in its last place): a gradient is a sum of two codes, exactly."""
    wc = _codes(out, n_in, 1)
    ws = torch.ones(out, device=DEV)
    dy = torch.zeros((batch, out), dtype=torch.float16, device=DEV)
    at = torch.from_numpy(np.random.default_rng(3).integers(0, out - 1, batch)).to(DEV)
    dy.scatter_(1, at[:, None], 1.0)
    dy[:, out - 1] = 2.0
    dx = I8Layer(wc, ws).grad_input(dy)
    t = _sample(batch, 200, 4)
    assert torch.equal(dx[t].float(), wc[at[t]].float() + 2 * wc[out - 1].float())


def test_gated_gradient_of_many_tokens():
    batch, out, n_in = 200000, 5600, 16       # g and u of more than 2^32 bytes each
    gate, up = _codes(out, n_in, 1), _codes(out, n_in, 2)
    block = I8Gated(I8Layer(gate, torch.ones(out, device=DEV)), I8Layer(up, torch.ones(out, device=DEV)), "silu")
    g = torch.full((batch, out), 64.0, device=DEV)
    u = torch.full((batch, out), 3.0, device=DEV)
    dh = torch.zeros((batch, out), dtype=torch.bfloat16, device=DEV)
    at = torch.from_numpy(np.random.default_rng(3).integers(0, out, batch)).to(DEV)
    dh.scatter_(1, at[:, None], 1.0)
    dx = block.grad_input(dh, g, u)
    t = _sample(batch, 200, 4)
    want = 3 * gate[at[t]].float() + 64 * up[at[t]].float()
    assert torch.equal(dx[t], want.to(torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_conversions(dtype):
    rows, cols = 140000, 16400                # 2.3e9 values
    codes = _codes(rows, cols, 1)
    codes[:, 7] = 127                         # every row reaches its scale
    scales = _scales(rows, 2)
    dense = i8_dequant(codes, scales, dtype)
    c2, s2 = i8_quantize(dense)
    t = _sample(rows, 300, 3)
    assert torch.equal(s2[t], scales[t]) and torch.equal(c2[t], codes[t])
    assert torch.equal(dense[t].double(), codes[t].double() * scales[t].double()[:, None])
