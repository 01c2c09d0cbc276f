"""Which kernels the int8 tests on the GPU run, held to the choice itself (csrc/i8_plan.hpp), without a GPU.

Whatever kernel a sweep over the sizes finds in use has to be run by one of test_gpu_i8_tiles.py's sizes. A
change of the modelled costs moves sizes between kernels: this is what then fails."""
import ctypes
import math
import random

import pytest

import i8_plans as plans
import test_gpu_i8_tiles as tiles
from additive_codebook_matmul_amd import load_library
from additive_codebook_matmul_amd.i8 import I8MatrixStruct

LISTS = {("product", False): tiles.PRODUCTS, ("product", True): tiles.GATED,
         ("grad", False): tiles.GRADS, ("grad", True): tiles.GATED_GRADS}
FEATURES = {"product": plans.product_features, "grad": plans.grad_features}


def _sweep(count, seed):
    """Sizes spread over their logarithms, half of the rows multiples of 8."""
    rng = random.Random(seed)

    def pick(high):
        return round(math.exp(rng.uniform(0, math.log(high))))
    for _ in range(count):
        out, n_in, batch = pick(40000), 16 * pick(1000), pick(5000)
        yield batch, max(8, out // 8 * 8) if rng.random() < 0.5 else out, n_in


def test_names_of_shapes():
    assert plans.shapes(False) == len(plans.TILES) == len(plans.RING)
    assert plans.shapes(True) == len(plans.GRAD_TILES) == len(plans.GRAD_RING)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", ["product", "grad"])
def test_every_kernel_in_use_is_tested(kind, gated):
    tested = set()
    for sizes in LISTS[kind, gated]:
        tested |= FEATURES[kind](*sizes, gated)
    missing = {}
    for sizes in _sweep(30000, 3):
        for f in FEATURES[kind](*sizes, gated) - tested:
            missing.setdefault(f, sizes)
    assert not missing


@pytest.mark.parametrize("kind,gated,names", [("product", False, plans.TILES), ("product", True, plans.TILES),
                                              ("grad", False, plans.GRAD_TILES), ("grad", True, plans.GRAD_TILES)])
def test_each_shape_is_tested_split_and_unsplit(kind, gated, names):
    """With one tile of tokens and with several, and with every remainder of a loop that turns."""
    found = set().union(*(FEATURES[kind](*sizes, gated) for sizes in LISTS[kind, gated]))
    for name in names:
        grids = {f[3:5] for f in found if f[:3] == (name, gated, "grid")}
        assert grids == {(s, t) for s in (False, True) for t in (False, True)}, name
        stages = (plans.RING if kind == "product" else plans.GRAD_RING)[name][0]
        assert {f[3] for f in found if f[:3] == (name, gated, "loop")} == set(range(stages)), name


def test_the_library_makes_these_choices():
    """Workspaces of the built library are those of the choices asked here."""
    lib = load_library()

    def asked(op, rows, cols, batch, pair):
        m, n = I8MatrixStruct(rows, cols, 4096, 4096), ctypes.c_int64(0)
        refs = [ctypes.byref(m)] * (2 if pair else 1)
        assert getattr(lib, f"aqlm_i8_{op}_workspace_size")(*refs, ctypes.c_int64(batch), ctypes.byref(n)) == 0
        return n.value
    for batch, rows, cols in _sweep(2000, 4):
        assert asked("gemm", rows, cols, batch, False) == plans.route(rows, cols, False, batch, False)["ws_bytes"]
        assert asked("gemm_quant", rows, cols, batch, False) == plans.route(rows, cols, False, batch)["ws_bytes"]
        assert asked("gated", rows, cols, batch, True) == plans.route(rows, cols, True, batch)["ws_bytes"]
        assert asked("grad_input", rows, cols, batch, False) == plans.grad(rows, cols, False, batch)["ws_bytes"]
        assert asked("gated_grad", rows, cols, batch, True) == plans.grad(rows, cols, True, batch)["ws_bytes"]
