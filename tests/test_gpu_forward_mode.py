"""Tensors that carry a forward-mode tangent: no operator computes with it, and none loses it in silence."""
import numpy as np
import pytest
import torch
from torch.autograd import forward_ad

from additive_codebook_matmul_amd import (I8Gated, I8Layer, MxLayer, i8_dequant, i8_quantize, mx_gemv_batched,
                                          mx_quantize)
from test_gpu_mx import DEV, HALVES

pytestmark = pytest.mark.gpu


def _dense(rows, cols, dtype, seed):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((rows, cols)).astype(np.float32)).to(DEV, dtype)


def _calls(dtype):
    """name: (operator of one tensor, shape)"""
    W = _dense(40, 64, dtype, 1)
    i8, mx = I8Layer.quantize(W), MxLayer.quantize(W)
    block = I8Gated(i8, i8)
    g = torch.ones((3, 40), device=DEV)
    return {"i8 forward": (i8.forward, 64), "i8 grad_input": (i8.grad_input, 40), "i8_quantize": (i8_quantize, 64),
            "gated forward": (block.forward, 64), "gated forward_saving": (block.forward_saving, 64),
            "gated grad_input": (lambda dh: block.grad_input(dh, g, g), 40),
            "mx forward": (mx.forward, 64), "mx forward_mx": (mx.forward_mx, 64), "mx gemv": (mx.gemv, 64),
            "mx batched": (lambda x: mx_gemv_batched([mx, mx], [x.detach(), x]), 64),
            "mx grad_input": (mx.grad_input, 40), "mx_quantize": (mx_quantize, 64)}


@pytest.mark.parametrize("recorded", [False, True])
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", ["i8 forward", "i8 grad_input", "i8_quantize", "gated forward", "gated forward_saving",
                                  "gated grad_input", "mx forward", "mx forward_mx", "mx gemv", "mx batched",
                                  "mx grad_input", "mx_quantize"])
def test_a_tangent_is_refused(name, dtype, recorded):
    call, cols = _calls(dtype)[name]
    x = _dense(3, cols, dtype, 2).requires_grad_(recorded)
    want = call(x)
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="tangent"):
            call(forward_ad.make_dual(x, torch.ones_like(x)))
        got = call(x)                                # a plain tensor passes inside of a level too
    for a, b in zip(want if isinstance(want, (tuple, list)) else [want], got if isinstance(got, (tuple, list)) else [got]):
        assert torch.equal(a, b) and a.requires_grad == b.requires_grad


@pytest.mark.parametrize("name", ["gemm_i8", "i8_dequant", "I8Layer"])
def test_a_tangent_of_scales_is_refused(name):
    codes, scales = i8_quantize(_dense(40, 64, torch.float16, 1))
    layer = I8Layer(codes, scales)
    call = {"gemm_i8": layer.gemm_i8, "i8_dequant": i8_dequant, "I8Layer": I8Layer}[name]
    with forward_ad.dual_level():
        call(codes, scales)
        with pytest.raises(ValueError, match="tangent"):
            call(codes, forward_ad.make_dual(scales, torch.ones_like(scales)))
