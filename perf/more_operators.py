"""Measured cases of the 8-bit integer operators.

An int8 matrix holds each row as whole numbers of [-127, 127] with one float32
scale: a row of activations is a token, a row of weights an output channel. The
operators are its quantisation and expansion, the linear layer whose activations
are quantised token by token, the gated feed-forward block act(gate(x)) * up(x) of
two such layers, and the gradients of both with respect to the activations
(straight through the quantisation), the weights being constants.

Shapes are the linear layers of Llama-2-7B (4096, 11008) and Llama-2-70B (8192,
28672), batches from one token to a prompt of 2048.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
ACTIVATIONS = ("silu", "gelu", "gelu_tanh")
LARGEST = 2048 * 11008 * 4096      # rows of activations x outputs x inputs


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the activations of three tokens, quantised for several layers that share
        # them: latency
        {"name": "convert_tokens", "op": "convert", "rows": 3, "cols": 4096, "dtype": "bf16"},
        # a Llama-2-70B gate or up projection quantised when it is loaded, and
        # expanded for a comparison with the dense one
        {"name": "convert_weight", "op": "convert", "rows": 28672, "cols": 8192, "dtype": "fp16"},
        # one token through a 70B down projection: the weights' bytes count
        {"name": "token_down_70b", "op": "product", "batch": 1, "out": 8192, "in": 28672,
         "dtype": "bf16"},
        # a ragged batch of sequences through a 7B down projection
        {"name": "batch_down", "op": "product", "batch": 77, "out": 4096, "in": 11008,
         "dtype": "fp16"},
        # a prompt of odd length through a 7B down projection
        {"name": "prompt_down", "op": "product", "batch": 1999, "out": 4096, "in": 11008,
         "dtype": "bf16"},
        # one token through the gate and up projections of a 7B block: latency
        {"name": "gated_token", "op": "gated", "batch": 1, "out": 11008, "in": 4096,
         "act": "silu", "dtype": "bf16"},
        # nineteen sequences' next tokens through those of a 70B block
        {"name": "gated_batch_70b", "op": "gated", "batch": 19, "out": 28672, "in": 8192,
         "act": "gelu", "dtype": "bf16"},
        # a prompt through those of a 7B block
        {"name": "gated_prompt", "op": "gated", "batch": 2048, "out": 11008, "in": 4096,
         "act": "silu", "dtype": "fp16"},
        # the backward pass of an adapter's training through a frozen projection
        {"name": "grad_up", "op": "grad", "batch": 2048, "out": 11008, "in": 4096,
         "dtype": "bf16"},
        # the same for a short ragged batch
        {"name": "grad_down", "op": "grad", "batch": 301, "out": 4096, "in": 11008,
         "dtype": "fp16"},
        # forward and backward of a frozen gated block inside of an adapter's training
        {"name": "gated_step", "op": "gated_step", "batch": 2048, "out": 11008, "in": 4096,
         "act": "silu", "dtype": "bf16"},
        # the same on one of eight parts of the block and a short ragged batch
        {"name": "gated_step_part", "op": "gated_step", "batch": 333, "out": 1376, "in": 4096,
         "act": "gelu_tanh", "dtype": "fp16"},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(("convert", "product", "product", "gated", "gated", "grad", "gated_step"))
    cols = 16 * _spread(rng, 8, 1792)
    if op == "convert":
        rows = min(_spread(rng, 1, 28672), 28672 * 8192 // cols)
        dtype = rng.choice(("fp16", "bf16", "fp32"))
        return {"op": op, "rows": rows // 2 + 1 if dtype == "fp32" else rows, "cols": cols, "dtype": dtype}
    out = min(_spread(rng, 64, 28672), 28672 * 8192 // cols)
    batch = min(_spread(rng, 1, 2048), max(1, LARGEST // (out * cols)))
    case = {"op": op, "batch": batch, "out": out, "in": cols, "dtype": rng.choice(("fp16", "bf16"))}
    if op in ("gated", "gated_step"):
        case["act"] = rng.choice(ACTIVATIONS)
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(shape, std, dtype, gen):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _activations(rows, cols, dtype, gen):
    """Normal values with a few wide channels, as the hidden states of a model have them."""
    x = torch.randn((rows, cols), generator=gen, device="cuda", dtype=torch.float32)
    wide = torch.rand(cols, generator=gen, device="cuda") < 0.005
    return (x * torch.where(wide, 12.0, 1.0)).to(dtype)


def _weights(out, cols, gen):
    """int8 weights and scales: normal ones with a spread of their own per row, quantised."""
    spread = torch.exp(0.3 * torch.randn((out, 1), generator=gen, device="cuda"))
    w = torch.randn((out, cols), generator=gen, device="cuda") * (0.02 * spread)
    codes, scales = _quantized(w)
    return codes.to(torch.int8), scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    state = {"op": op, "dtype": dtype, "act": case.get("act")}
    if op == "convert":
        if case["rows"] >= 256:
            state["x"] = _normal((case["rows"], case["cols"]), 0.02, dtype, gen)
        else:
            state["x"] = _activations(case["rows"], case["cols"], dtype, gen)
        return state
    state["weights"] = [_weights(case["out"], case["in"], gen)
                        for _ in range(2 if op in ("gated", "gated_step") else 1)]
    if op != "grad":
        state["x"] = _activations(case["batch"], case["in"], dtype, gen)
    if op in ("grad", "gated_step"):
        state["dy"] = _normal((case["batch"], case["out"]), 0.01, dtype, gen)
    if own:
        from additive_codebook_matmul_amd import I8Gated, I8Layer
        layers = [I8Layer(codes, scales) for codes, scales in state["weights"]]
        state["layer"] = layers[0] if len(layers) == 1 else I8Gated(*layers, case["act"])
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _quantized(x):
    """(whole numbers [rows, cols], float32 scales [rows]) of x: the row's largest
    magnitude stands for 127, values go to the nearest multiple of a 127th of it,
    ties to the even one. (Divided in 64 bits: near a tie 32 would decide wrongly.)"""
    top = x.abs().amax(dim=1, keepdim=True)
    safe = torch.where(top == 0, torch.ones_like(top), top).double()
    codes = torch.round(x.double() * 127.0 / safe)
    return codes.float(), (top.float() / 127.0).squeeze(1)


def _product(q, s, weights):
    """float32 Q(x) . W^T of codes and scales."""
    codes, scales = weights
    return (q @ codes.float().t()) * s.unsqueeze(1) * scales


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        c = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * c, c + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    k, a = 2.0 * math.sqrt(2.0 / math.pi), 0.044715
    s = 1.0 / (1.0 + torch.exp(-k * (g + a * g * g * g)))
    return g * s, s + g * s * (1.0 - s) * k * (1.0 + 3.0 * a * g * g)


def _back(dy, weights):
    codes, scales = weights
    return (dy * scales) @ codes.float()


def _plain(state):
    op, dtype = state["op"], state["dtype"]
    if op == "convert":
        codes, scales = _quantized(state["x"])
        return {"values": (codes * scales.unsqueeze(1)).to(dtype), "scales": scales}
    if op == "grad":
        return _back(state["dy"].float(), state["weights"][0]).to(dtype)
    q, s = _quantized(state["x"])
    if op == "product":
        return _product(q, s, state["weights"][0]).to(dtype)
    gate, up = state["weights"]
    g, u = _product(q, s, gate), _product(q, s, up)
    a, slope = _act(g, state["act"])
    h = (a * u).to(dtype)
    if op == "gated":
        return h
    dy = state["dy"].float()
    return {"h": h, "dx": (_back(dy * u * slope, gate) + _back(dy * a, up)).to(dtype)}


# ---------------------------------------------------------------------------
# the framework's operators
# ---------------------------------------------------------------------------
def _framework(state):
    from additive_codebook_matmul_amd import i8_dequant, i8_quantize
    op = state["op"]
    if op == "convert":
        codes, scales = i8_quantize(state["x"])
        return {"values": i8_dequant(codes, scales, dtype=state["dtype"]), "scales": scales}
    layer = state["layer"]
    if op == "grad":
        return layer.grad_input(state["dy"])
    if op != "gated_step":
        return layer.forward(state["x"])
    x = state["x"].detach().requires_grad_()
    h = layer.forward(x)
    (dx,) = torch.autograd.grad(h, x, state["dy"])
    return {"h": h.detach(), "dx": dx}


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "convert":  # x read; values and scales written
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * size + case["rows"] * 4, "flops": 4 * n}
    b, o, i = case["batch"], case["out"], case["in"]
    layers = 1 if case["op"] in ("product", "grad") else 2
    weights = layers * (o * i + 4 * o)
    if case["op"] == "gated_step":  # x, the incoming gradient, h and dx
        return {"bytes": weights + 2 * (2 * b * i + 2 * b * o), "flops": 2 * 2 * layers * b * o * i}
    return {"bytes": weights + 2 * (b * i + b * o), "flops": 2 * layers * b * o * i}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_rows(x):
    """Codes and scales of x: n is the code of v where |127 v / top - n| is least,
    and even where two are as near."""
    v = x.double()
    top = v.abs().max(dim=1, keepdim=True).values
    r = torch.where(top > 0, v.abs() * 127 / torch.where(top > 0, top, torch.ones_like(top)),
                    torch.zeros_like(v))
    low = torch.floor(r)
    rest = r - low
    odd = (low.long() & 1).double()
    n = low + torch.where(rest == 0.5, odd, (rest > 0.5).double())
    return torch.copysign(n, v), top / 127


def _exact_act(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if act == "gelu":
        phi = torch.special.ndtr(g)
        return g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    near = torch.sigmoid(2 * c * (g + 0.044715 * g ** 3))    # (1 + t) / 2, exact far below zero too
    return g * near, near + g / 2 * (1 - t * t) * c * (1 + 0.134145 * g * g)


def exact(case, seed):
    state = prepare(case, seed)
    op = state["op"]
    if op == "convert":
        n, scale = _exact_rows(state["x"])
        return {"values": n * scale, "scales": scale.squeeze(1)}
    dense = [codes.double() * scales.double().unsqueeze(1) for codes, scales in state["weights"]]
    if op == "grad":
        return state["dy"].double() @ dense[0]
    n, scale = _exact_rows(state["x"])
    sums = [(n * scale) @ w.t() for w in dense]
    if op == "product":
        return sums[0]
    a, slope = _exact_act(sums[0], state["act"])
    if op == "gated":
        return a * sums[1]
    dy = state["dy"].double()
    return {"h": a * sums[1], "dx": (dy * sums[1] * slope) @ dense[0] + (dy * a) @ dense[1]}
