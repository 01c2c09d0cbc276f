"""Microscaled layers under autograd: an activation that requires a gradient gets it through the
frozen weights. Whole numbers throughout, so that every gradient is exact in both types."""
import numpy as np
import pytest
import torch

from additive_codebook_matmul_amd import MxLayer, mx_gemv_batched
from oracle import mx_oracle as MO
from test_gpu_mx import DEV, HALVES, dev, rounded, same

pytestmark = pytest.mark.gpu


def _weights(out, n_in, seed):
    """Sparse weights of 1 and -1: sums stay whole and small."""
    rng = np.random.default_rng(seed)
    codes = np.where(rng.random((out, n_in)) < 0.2, rng.choice([2, 10], (out, n_in)), 0).astype(np.uint8)
    packed, scales = MO.pack(codes), np.full((out, n_in // 32), 127, dtype=np.uint8)
    return MxLayer(dev(packed), dev(scales)), MO.dequant(packed, scales)


def _whole(rows, cols, seed):
    return np.random.default_rng(seed).integers(-1, 2, (rows, cols)).astype(np.float64)


def _leaf(a, dtype):
    return rounded(a, dtype).to(DEV).requires_grad_()


CALLS = {"forward": lambda L, x: L.forward(x), "gemm": lambda L, x: L.gemm(x),
         "forward_mx": lambda L, x: L.forward_mx(x), "gemv": lambda L, x: L.gemv(x),
         "batched": lambda L, x: mx_gemv_batched([L], [x])[0]}


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("call,batch,out,n_in",
                         [(c, *s) for c in CALLS for s in [(1, 40, 64), (6, 37, 96), (50, 131, 160)]
                          if s[0] <= 8 or c not in ("gemv", "batched")])
def test_gradient_of_each_product(call, batch, out, n_in, dtype):
    layer, w = _weights(out, n_in, batch)
    x = _leaf(_whole(batch, n_in, 1), dtype)
    y = CALLS[call](layer, x)
    assert y.requires_grad and y.dtype == dtype
    same(y.detach(), rounded(_whole(batch, n_in, 1) @ w.T, dtype))
    dy = _whole(batch, out, 2)
    y.backward(rounded(dy, dtype).to(DEV))
    same(x.grad, rounded(dy @ w, dtype))
    with torch.no_grad():
        plain = CALLS[call](layer, x)
    assert not plain.requires_grad and torch.equal(plain, y)


@pytest.mark.parametrize("dtype", HALVES)
def test_gradient_by_differences(dtype):
    layer, w = _weights(40, 64, 3)
    a, dy = _whole(5, 64, 4), _whole(5, 40, 5)
    x = _leaf(a, dtype)
    (grad,) = torch.autograd.grad(layer.forward(x), x, rounded(dy, dtype).to(DEV))
    with torch.no_grad():
        for i in range(0, 64, 7):
            step = np.zeros_like(a)
            step[:, i] = 1
            up = layer.forward(_leaf(a + step, dtype)).cpu().double().numpy()
            down = layer.forward(_leaf(a - step, dtype)).cpu().double().numpy()
            assert np.array_equal(((up - down) * dy).sum(1) / 2, grad[:, i].cpu().double().numpy())


@pytest.mark.parametrize("dtype", HALVES)
def test_an_adapter_beside_a_frozen_layer(dtype):
    """y = W x + B A x, below it another trained matrix: every gradient has the frozen layer's part."""
    layer, w = _weights(48, 64, 1)
    a, t = _whole(7, 32, 2), _whole(64, 32, 3)
    A, B = _whole(4, 64, 4), _whole(48, 4, 5)
    pa, pb, pt = _leaf(A, dtype), _leaf(B, dtype), _leaf(t, dtype)
    h = rounded(a, dtype).to(DEV) @ pt.t()
    y = layer.forward(h) + (h @ pa.t()) @ pb.t()
    dy = _whole(7, 48, 6)
    y.backward(rounded(dy, dtype).to(DEV))
    dh = dy @ w + (dy @ B) @ A
    # steps of the plain products round to the type: their own tests' tolerance, half a step each,
    # three of them before the last, which is a sum of 7 terms
    bound = (np.abs(dy) @ np.abs(w) + np.abs(dy) @ np.abs(B) @ np.abs(A)).T @ np.abs(a)
    tol = 4 * torch.finfo(dtype).eps / 2 * bound * (1 + torch.finfo(dtype).eps)
    assert (np.abs(pt.grad.cpu().double().numpy() - dh.T @ a) <= tol).all()
    assert pa.grad is not None and pb.grad is not None


@pytest.mark.parametrize("dtype", HALVES)
def test_grouped_layers_add_to_a_shared_input(dtype):
    """Query, key and value of one input; one result unused, one gradient given twice."""
    parts = [_weights(40, 64, k) for k in range(3)] + [_weights(24, 96, 3)]
    layers = [p[0] for p in parts]
    x, other = _leaf(_whole(5, 64, 7), dtype), _leaf(_whole(5, 96, 8), dtype)
    ys = mx_gemv_batched(layers, [x, x, x, other])
    assert all(y.requires_grad for y in ys)
    dy = [_whole(5, y.shape[1], 9 + k) for k, y in enumerate(ys)]
    d = [rounded(v, dtype).to(DEV) for v in dy]
    loss = (ys[0] * d[0]).sum() + (ys[2] * d[2]).sum() + (ys[3] * d[3]).sum()
    gx, go = torch.autograd.grad(loss, (x, other), retain_graph=True)
    same(gx, rounded(dy[0] @ parts[0][1] + dy[2] @ parts[2][1], dtype))
    same(go, rounded(dy[3] @ parts[3][1], dtype))
    again = torch.autograd.grad(loss, (x, other))
    assert torch.equal(again[0], gx) and torch.equal(again[1], go)
    ys[0].add_(1)                                     # results may be changed in place
    frozen = mx_gemv_batched(layers[:2], [x.detach(), x.detach()])
    assert not frozen[0].requires_grad
    mixed = mx_gemv_batched([layers[0], layers[3]], [x.detach(), other])
    (go,) = torch.autograd.grad(mixed[1], other, d[3])
    same(go, rounded(dy[3] @ parts[3][1], dtype))


@pytest.mark.parametrize("dtype", HALVES)
def test_gradients_as_autograd_hands_them_over(dtype):
    """Expanded, transposed, and off alignment (odd rows of a part of a larger gradient)."""
    layer, w = _weights(37, 64, 2)
    a = _whole(6, 64, 3)
    x = _leaf(a, dtype)
    layer.forward(x).sum().backward()
    same(x.grad, rounded(np.ones((6, 37)) @ w, dtype))
    x = _leaf(a, dtype)
    d = _whole(37, 6, 4)
    layer.forward(x).t().backward(rounded(d, dtype).to(DEV))
    same(x.grad, rounded(d.T @ w, dtype))
    x, z = _leaf(a, dtype), _leaf(_whole(1, 64, 5), dtype)
    d = _whole(7, 37, 6)
    torch.cat([layer.forward(z), layer.forward(x)]).backward(rounded(d, dtype).to(DEV))
    same(x.grad, rounded(d[1:] @ w, dtype))
    same(z.grad, rounded(d[:1] @ w, dtype))
    empty = torch.empty((0, 64), dtype=dtype, device=DEV, requires_grad=True)
    layer.forward(empty).sum().backward()
    assert empty.grad.shape == (0, 64)


def test_what_autograd_cannot_record_is_refused():
    layer, _ = _weights(40, 64, 1)
    x = _leaf(_whole(4, 64, 1), torch.float16)
    out = torch.empty((4, 40), dtype=torch.float16, device=DEV)
    for call in (lambda: layer.gemm(x, out=out), lambda: layer.forward_mx(x, out=out),
                 lambda: layer.gemv(x, out=out), lambda: mx_gemv_batched([layer], [x], [out])):
        with pytest.raises(ValueError, match="out"):
            call()
        with torch.no_grad():
            call()
    with pytest.raises(ValueError):                   # the arguments' own checks come first
        layer.forward(x[:, :32])
    (g,) = torch.autograd.grad(layer.forward(x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


@pytest.mark.parametrize("dtype", HALVES)
def test_a_captured_step(dtype):
    """Forward and backward in one graph, replayed on new activations between eager steps."""
    layer, w = _weights(72, 96, 1)
    static, d = rounded(_whole(9, 96, 1), dtype).to(DEV), rounded(_whole(9, 72, 2), dtype).to(DEV)

    def step():
        x = static.detach().requires_grad_()          # a leaf of the step's own
        y = layer.forward(x)
        (g,) = torch.autograd.grad(y, x, d)
        return y.detach(), g
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, dx = step()
    for k in range(4):
        a, b = _whole(9, 96, 10 + k), _whole(9, 72, 20 + k)
        static.copy_(rounded(a, dtype))
        d.copy_(rounded(b, dtype))
        y.zero_()
        dx.zero_()
        g.replay()
        torch.cuda.synchronize()
        same(y, rounded(a @ w.T, dtype))
        same(dx, rounded(b @ w, dtype))
        ey, edx = step()
        assert torch.equal(ey, y) and torch.equal(edx, dx)
    del g
    torch.cuda.empty_cache()
