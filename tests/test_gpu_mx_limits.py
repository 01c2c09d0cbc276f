"""The microscaled products and the input gradient at the largest rows, columns and batch that they
take, 2^21 each. Sums are whole multiples of 2^-3 below 2^21: exact in any order."""
import pytest
import torch

from additive_codebook_matmul_amd import MxLayer, mx_quantize
from oracle import mx_oracle as MO
from test_gpu_mx import DEV, HALVES

pytestmark = pytest.mark.gpu

MOST = 1 << 21


def _codes(rows, cols, gen):
    codes = torch.randint(0, 256, (rows, cols // 2), generator=gen, device=DEV, dtype=torch.uint8)
    return codes, torch.randint(125, 130, (rows, cols // 32), generator=gen, device=DEV, dtype=torch.uint8)


def _whole(rows, cols, gen, dtype):
    return torch.randint(-2, 3, (rows, cols), generator=gen, device=DEV, dtype=torch.int8).to(dtype)


def _gen(seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return gen


def _check(layer, x, want):
    """want: float32, exact. (Activations of whole numbers up to 2 are microscaled exactly.)"""
    want = want.to(x.dtype)
    assert torch.equal(layer.gemm(x), want)
    assert torch.equal(layer.gemm_mx(*mx_quantize(x), x.dtype), want)
    assert torch.equal(layer.forward_mx(x, "ceil"), want)
    if x.shape[0] <= 8:
        assert torch.equal(layer.gemv(x), want)


@pytest.mark.parametrize("dtype", HALVES)
def test_most_columns(dtype):
    gen, out, terms = _gen(1), 40, 16
    at = torch.randint(0, MOST // terms, (out, terms), generator=gen, device=DEV)
    at += torch.arange(terms, device=DEV) * (MOST // terms)
    at[:, 0], at[:, -1] = 0, MOST - 1
    code = torch.randint(1, 16, (out, terms), generator=gen, device=DEV, dtype=torch.uint8)
    codes = torch.zeros((out, MOST // 2), dtype=torch.uint8, device=DEV)
    codes.scatter_(1, at // 2, code << (4 * (at % 2)).to(torch.uint8))
    scales = torch.randint(125, 130, (out, MOST // 32), generator=gen, device=DEV, dtype=torch.uint8)
    layer = MxLayer(codes, scales)
    value = torch.from_numpy(MO.E2M1).float().to(DEV)[code.long()]
    w = value * torch.exp2(scales.gather(1, at // 32).float() - 127)
    for batch in (1, 2, 5, 12, 40, 100, 300):
        x = _whole(batch, MOST, gen, dtype)
        _check(layer, x, torch.stack([(x[:, at[o]].float() * w[o]).sum(1) for o in range(out)], 1))
    dy = _whole(3, out, gen, dtype)
    dx = layer.grad_input(dy)
    want = torch.zeros((3, MOST), device=DEV)
    for o in range(out):
        want[:, at[o]] += dy[:, o, None].float() * w[o]
    assert torch.equal(dx, want.to(dtype))


@pytest.mark.parametrize("dtype", HALVES)
def test_most_rows(dtype):
    gen, n_in = _gen(2), 64
    layer = MxLayer(*_codes(MOST, n_in, gen))
    w = layer.dequant(torch.float32)
    for batch in (1, 2, 5, 12, 40):
        x = _whole(batch, n_in, gen, dtype)
        _check(layer, x, x.float() @ w.t())
    at = torch.tensor([0, 1, 255, 256, MOST // 2, MOST - 257, MOST - 2, MOST - 1], device=DEV)
    for batch in (1, 40, 130):
        dy = torch.zeros((batch, MOST), dtype=dtype, device=DEV)
        dy[:, at] = _whole(batch, len(at), gen, dtype)
        assert torch.equal(layer.grad_input(dy), (dy[:, at].float() @ w[at]).to(dtype))


@pytest.mark.parametrize("dtype", HALVES)
def test_largest_batch(dtype):
    gen, out, n_in = _gen(3), 40, 64
    layer = MxLayer(*_codes(out, n_in, gen))
    w = layer.dequant(torch.float32)
    x = _whole(MOST, n_in, gen, dtype)
    _check(layer, x, x.float() @ w.t())
    dy = _whole(MOST, out, gen, dtype)
    assert torch.equal(layer.grad_input(dy), (dy.float() @ w).to(dtype))
    odd = MxLayer(layer.codes[:37].contiguous(), layer.scales[:37].contiguous())   # rows padded first
    assert torch.equal(odd.grad_input(dy[:, :37].contiguous()), (dy[:, :37].float() @ w[:37]).to(dtype))
