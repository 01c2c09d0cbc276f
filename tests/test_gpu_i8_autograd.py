"""int8 layers and gated blocks as a program uses them: under autograd, chained to a whole
feed-forward block, in a captured graph, on another stream; and gradients against differences."""
import numpy as np
import pytest
import torch

from additive_codebook_matmul_amd import I8Gated, I8Layer, i8_quantize
from oracle import i8_oracle as IO
from test_gpu_i8 import (ACTS, activations, gated_case, gated_tolerance, grad_tolerance, half, layer_of, product,
                         small_weights, weights, whole)
from test_gpu_mx import DEV, HALVES, dev, rounded, same

pytestmark = pytest.mark.gpu


def _leaf(a, dtype):
    return rounded(a, dtype).to(DEV).requires_grad_()


def _unit_rows(batch, n_in, seed):
    """Whole activations whose rows reach 127: their codes are themselves, their scale 1."""
    x = np.random.default_rng(seed).integers(-3, 4, (batch, n_in)).astype(np.float64)
    x[:, 0] = 127
    return x


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", [(1, 40, 64), (6, 37, 96), (50, 131, 160), (200, 260, 272)])
def test_gradient_of_a_layer(batch, out, n_in, dtype):
    w = small_weights(out, n_in, batch)
    layer = layer_of(w)
    a = _unit_rows(batch, n_in, 1)
    x = _leaf(a, dtype)
    y = layer.forward(x)
    assert y.requires_grad and y.dtype == dtype
    same(y.detach(), half(product(x.detach().cpu(), w, dtype), dtype))
    dy = whole(batch, out, 2)
    y.backward(rounded(dy, dtype).to(DEV))
    same(x.grad, half(IO.back(dy * w[1][None, :], w[0])[0], dtype))
    with torch.no_grad():
        plain = layer.forward(x)
    assert not plain.requires_grad and torch.equal(plain, y)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,out,n_in", [(1, 40, 64), (7, 37, 96), (90, 131, 160)])
def test_gradient_of_a_gated_block(batch, out, n_in, dtype, act):
    gate, up, x = gated_case(batch, out, n_in, dtype)
    block = I8Gated(layer_of(gate), layer_of(up), act)
    leaf = x.to(DEV).requires_grad_()
    h = block.forward(leaf)
    with torch.no_grad():
        assert torch.equal(block.forward(leaf), h)
    dh = rounded(np.random.default_rng(3).standard_normal((batch, out)) * 0.1, dtype).to(DEV)
    (dx,) = torch.autograd.grad(h, leaf, dh, retain_graph=True)
    _, g, u = block.forward_saving(leaf)
    assert torch.equal(dx, block.grad_input(dh, g, u))
    (again,) = torch.autograd.grad(h, leaf, dh)
    assert torch.equal(again, dx)
    assert dx.shape == x.shape and dx.dtype == dtype and bool(torch.isfinite(dx).all())


@pytest.mark.parametrize("dtype", HALVES)
def test_gradient_of_a_layer_by_differences(dtype):
    w = small_weights(40, 64, 3)
    layer, a, dy = layer_of(w), _unit_rows(5, 64, 4), whole(5, 40, 5)
    x = _leaf(a, dtype)
    (grad,) = torch.autograd.grad(layer.forward(x), x, rounded(dy, dtype).to(DEV))
    codes, scales = i8_quantize(x.detach())
    assert torch.equal(codes.to(dtype), x.detach()) and bool((scales == 1).all())
    for i in range(1, 64, 7):       # (column 0 holds the rows' largest values)
        up, down = codes.clone(), codes.clone()
        up[:, i] += 1
        down[:, i] -= 1
        # float32-exact products: differences of the exact sums
        d = (product_of(up, scales, w) - product_of(down, scales, w)) / 2
        want = (d * dy).sum(1)
        got = grad[:, i].cpu().double().numpy()
        assert np.array_equal(half(want, dtype).double().numpy(), got)


def product_of(codes, scales, w):
    return IO.value(IO.sums(codes.cpu().numpy(), w[0]), w[1], scales.cpu().numpy()).astype(np.float64)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", HALVES)
def test_gradient_of_a_gated_block_by_differences(dtype, act):
    """h is taken from the block's float32 g and u at x + e_i and x - e_i. With a and b the steps of g and
    u, the central difference is off by at most |act'''| a^3 |u| / 6 + |act''| a^2 b / 2 (|act''| < 1.2,
    |act'''| < 2 for all three) and by the roundings of g and u, three of 2^-24 each."""
    batch, out, n_in = 4, 40, 64
    rng = np.random.default_rng(7)
    gate, up = ((rng.integers(-127, 128, (out, n_in)).astype(np.int8), np.full(out, np.float32(2.0 ** -13)))
                for _ in range(2))
    block = I8Gated(layer_of(gate), layer_of(up), act)
    a, dh = _unit_rows(batch, n_in, 8), rounded(rng.standard_normal((batch, out)), dtype)
    x = _leaf(a, dtype)
    _, g, u = block.forward_saving(x)
    grad = block.grad_input(dh.to(DEV), g, u).cpu().double().numpy()
    d64, g0, u0 = dh.double().numpy(), g.cpu().double().numpy(), u.cpu().double().numpy()

    def value(shift):
        _, gs, us = block.forward_saving(_leaf(a + shift, dtype))
        return IO.act(gs.cpu().double().numpy(), act)[0] * us.cpu().double().numpy()
    tg, tu = IO.gated_terms(g0, u0, d64, gate[1].astype(np.float64), up[1].astype(np.float64), act)
    both, codes = np.concatenate([tg, tu], axis=1), np.concatenate([gate[0], up[0]])
    rounding = grad_tolerance(both, IO.back(both, codes)[0], codes, dtype)
    for i in range(1, n_in, 5):
        step = np.zeros_like(a)
        step[:, i] = 1
        slope = ((value(step) - value(-step)) / 2 * d64).sum(1)
        da, db = (np.abs(w[0][:, i].astype(np.float64)) * w[1][0] for w in (gate, up))
        off = 2 * da ** 3 * (np.abs(u0) + db) / 6 + 1.2 * da ** 2 * db / 2
        off = off + 4 * 2.0 ** -24 * (1.13 * np.abs(g0) * np.abs(u0) + np.abs(g0) + np.abs(u0) + 1)
        tol = (np.abs(d64) * off).sum(1) + rounding[:, i]
        assert (np.abs(slope - grad[:, i]) <= tol).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,width,inner", [(1, 256, 688), (3, 128, 352), (19, 256, 688), (150, 128, 1376)])
def test_a_whole_feed_forward_block(batch, width, inner, dtype, act):
    """down(act(gate(x)) * up(x)) and its gradient through all three layers, each step against the oracle
    on the step's own inputs."""
    gate, up, x = gated_case(batch, inner, width, dtype)
    down = weights(width, inner, 9)
    down[1][:] *= np.float32(16 / np.sqrt(inner))
    block, last = I8Gated(layer_of(gate), layer_of(up), act), layer_of(down)
    leaf = x.to(DEV).requires_grad_()
    h = block.forward(leaf)
    h.retain_grad()
    y = last.forward(h)
    dy = rounded(np.random.default_rng(5).standard_normal((batch, width)) * 0.05, dtype)
    y.backward(dy.to(DEV))
    g, u = product(x, gate, dtype), product(x, up, dtype)
    a, _ = IO.act(g, act)
    ref, got = a * u.astype(np.float64), h.detach().cpu().double().numpy()
    # (from half a step above the type's largest number on, 2^16 (1 - 2^-12) for float16, a
    # result is an infinity, and its token's result of the next layer NaN)
    inside = np.abs(ref) < torch.finfo(dtype).max
    far = np.abs(np.where(inside, got - ref, 0))
    assert (far <= gated_tolerance(g.astype(np.float64), u, a, dtype)).all()
    beyond = np.abs(ref) >= torch.finfo(dtype).max * (1 + torch.finfo(dtype).eps)
    assert (got[beyond] == np.copysign(np.inf, ref[beyond])).all()
    same(y.detach(), half(product(h.detach().cpu(), down, dtype), dtype))
    terms = dy.double().numpy() * down[1].astype(np.float64)[None, :]
    ref = IO.back(terms, down[0])[0]
    dh = h.grad.cpu()
    assert (np.abs(dh.double().numpy() - ref) <= grad_tolerance(terms, ref, down[0], dtype)).all()
    tg, tu = IO.gated_terms(g.astype(np.float64), u.astype(np.float64), dh.double().numpy(),
                            gate[1].astype(np.float64), up[1].astype(np.float64), act)
    both, codes = np.concatenate([tg, tu], axis=1), np.concatenate([gate[0], up[0]])
    ref = IO.back(both, codes)[0]
    d64, g64 = np.abs(dh.double().numpy()), np.abs(g.astype(np.float64))
    slack = 64 * 2.0 ** -24 * (
        IO.back(d64 * np.abs(u) * (1 + g64 ** 2) * gate[1].astype(np.float64)[None, :], np.abs(gate[0].astype(np.int16)))[0]
        + IO.back(d64 * g64 * up[1].astype(np.float64)[None, :], np.abs(up[0].astype(np.int16)))[0])
    assert (np.abs(leaf.grad.cpu().double().numpy() - ref) <= grad_tolerance(both, ref, codes, dtype) + slack).all()


@pytest.mark.parametrize("dtype", HALVES)
def test_joined_layers_give_their_parts(dtype):
    """Query, key and value joined along `out` are one layer: each part's bits are its own layer's."""
    parts = [weights(48, 96, k) for k in range(3)]
    joined = I8Layer(dev(np.concatenate([p[0] for p in parts])), dev(np.concatenate([p[1] for p in parts])))
    for batch in (1, 4, 30, 130):
        x = activations(batch, 96, dtype, batch).to(DEV)
        ys = joined.forward(x).split(48, dim=1)
        for y, p in zip(ys, parts):
            assert torch.equal(y, layer_of(p).forward(x))


@pytest.mark.parametrize("dtype", HALVES)
def test_gradients_as_autograd_hands_them_over(dtype):
    """Expanded, transposed, and off alignment (odd rows of a part of a larger gradient)."""
    w = small_weights(37, 64, 2)
    layer, a = layer_of(w), _unit_rows(6, 64, 3)
    x = _leaf(a, dtype)
    layer.forward(x).sum().backward()
    same(x.grad, half(IO.back(np.ones((6, 37)) * w[1][None, :], w[0])[0], dtype))
    x, d = _leaf(a, dtype), whole(37, 6, 4)
    layer.forward(x).t().backward(rounded(d, dtype).to(DEV))
    same(x.grad, half(IO.back(d.T * w[1][None, :], w[0])[0], dtype))
    block = I8Gated(layer, layer_of(small_weights(37, 64, 3)))
    x, z, d = _leaf(a, dtype), _leaf(_unit_rows(1, 64, 5), dtype), rounded(whole(7, 37, 6), dtype).to(DEV)
    torch.cat([block.forward(z), block.forward(x)]).backward(d)
    for leaf, part in ((z, d[:1]), (x, d[1:])):
        _, g, u = block.forward_saving(leaf)
        assert torch.equal(leaf.grad, block.grad_input(part.clone(), g, u))
    x = _leaf(a, dtype)
    block.forward(x).sum().backward()
    _, g, u = block.forward_saving(x)
    assert torch.equal(x.grad, block.grad_input(torch.ones((6, 37), dtype=dtype, device=DEV), g, u))
    empty = torch.empty((0, 64), dtype=dtype, device=DEV, requires_grad=True)
    (layer.forward(empty).sum() + block.forward(empty).sum()).backward()
    assert empty.grad.shape == (0, 64)


def test_what_autograd_cannot_record_is_refused():
    layer = layer_of(weights(40, 64, 1))
    block = I8Gated(layer, layer)
    x = _leaf(_unit_rows(4, 64, 1), torch.float16)
    out = torch.empty((4, 40), dtype=torch.float16, device=DEV)
    for call in (lambda: layer.forward(x, out=out), lambda: block.forward(x, out=out)):
        with pytest.raises(ValueError, match="out"):
            call()
        with torch.no_grad():
            call()
    for call in (layer.forward, block.forward):
        with pytest.raises(ValueError):                   # the arguments' own checks come first
            call(x[:, :32])
        (g,) = torch.autograd.grad(call(x).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            g.sum().backward()
    saved = block.forward_saving(x)
    assert not any(t.requires_grad for t in saved)


def _bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,width,inner", [(1, 96, 80), (9, 96, 80), (40, 512, 1008), (150, 1024, 2048)])
def test_a_captured_step(batch, width, inner, dtype):
    """A whole block's forward and backward in one graph, replayed on new activations between eager steps."""
    gate, up, _ = gated_case(batch, inner, width, dtype)
    down = weights(width, inner, 9)
    block, last = I8Gated(layer_of(gate), layer_of(up)), layer_of(down)
    static, d = activations(batch, width, dtype, 1).to(DEV), activations(batch, width, dtype, 2).to(DEV)

    def step():
        x = static.detach().requires_grad_()          # a leaf of the step's own
        y = last.forward(block.forward(x))
        (g,) = torch.autograd.grad(y, x, d)
        return y.detach(), g
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dx = step()
    for k in range(4):
        static.copy_(activations(batch, width, dtype, 10 + k))
        d.copy_(activations(batch, width, dtype, 20 + k))
        y.zero_()
        dx.zero_()
        graph.replay()
        torch.cuda.synchronize()
        ey, edx = step()
        assert _bits(ey, y) and _bits(edx, dx)        # (tokens beyond float16 are NaN in both)
    del graph
    torch.cuda.empty_cache()


@pytest.mark.parametrize("batch", [2, 20, 300])
def test_calls_on_two_streams_at_once(batch):
    """Workspaces of overlapping calls are their own."""
    dtype = torch.bfloat16
    w = weights(1000, 2048, 1)
    layer = layer_of(w)
    xs = [activations(batch, 2048, dtype, k).to(DEV) for k in range(2)]
    dys = [activations(batch, 1000, dtype, k + 2).to(DEV) for k in range(2)]
    want = [(layer.forward(x), layer.grad_input(dy)) for x, dy in zip(xs, dys)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append((layer.forward(xs[k]), layer.grad_input(dys[k])))
    torch.cuda.synchronize()
    for k in range(2):
        for y, dx in got[k]:
            assert torch.equal(y, want[k][0]) and torch.equal(dx, want[k][1])


def test_repeated_calls_same_bits():
    dtype = torch.float16
    gate, up, x = gated_case(77, 1100, 4096, dtype)
    block, x = I8Gated(layer_of(gate), layer_of(up), "gelu"), x.to(DEV)
    h, g, u = block.forward_saving(x)
    dx = block.grad_input(h, g, u)
    for _ in range(5):
        h2, g2, u2 = block.forward_saving(x)
        assert torch.equal(h2, h) and torch.equal(g2, g) and torch.equal(u2, u)
        assert _bits(block.grad_input(h, g, u), dx)   # (the gradient h has infinities, dx NaN then)
