"""The int8 operators' choice of kernels, asked on the host: csrc/i8_plan.hpp compiled by itself.

`route` and `grad` return what a product or a gradient of given sizes is done with; the tests of the tile
kernels state which kernels their sizes reach, and a test without a GPU holds them to it."""
import ctypes
import os
import shutil
import subprocess
import tempfile

from additive_codebook_matmul_amd import build

KINDS = ("rows", "skinny", "tiles")
TILES = ("Large", "Wide", "Middle", "Half", "Small", "Slim", "Least")
GRAD_TILES = ("Large", "Half", "Small", "Deep")

SOURCE = """
#include "i8_plan.hpp"
using namespace aqlm;
static void plan_of(const I8Plan &p, int64_t *out) {
  out[0] = p.shape; out[1] = p.splits; out[2] = p.steps_per_split; out[3] = p.across; out[4] = p.tok_tiles;
}
extern "C" {
void i8_test_route(int64_t rows, int64_t cols, int gated, int64_t batch, int quant, int64_t *out) {
  const I8Route r = i8_route(rows, cols, gated != 0, batch, quant != 0);
  plan_of(r.plan, out);
  out[5] = r.kind; out[6] = r.inside; out[7] = r.ws_bytes;
}
void i8_test_grad(int64_t rows, int64_t cols, int gated, int64_t batch, int64_t *out) {
  const I8Plan p = i8_grad_plan(rows, cols, gated != 0, batch);
  plan_of(p, out);
  out[7] = i8_grad_ws_bytes(rows, gated != 0, batch, p);
}
int i8_test_shapes(int grad) {
  return (int)(grad ? sizeof(i8_grad::kCosts) / sizeof(i8_grad::kCosts[0]) : sizeof(i8_tile::kCosts) / sizeof(i8_tile::kCosts[0]));
}
}
"""

_lib = None


def _load():
    global _lib
    if _lib is None:
        with tempfile.TemporaryDirectory() as tmp:
            source, out = os.path.join(tmp, "plans.cpp"), os.path.join(tmp, "plans.so")
            with open(source, "w") as f:
                f.write(SOURCE)
            cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
            subprocess.run([cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-I", build.CSRC, source, "-o", out], check=True)
            _lib = ctypes.CDLL(out)
    return _lib


def route(rows, cols, gated, batch, quant=True):
    """What a layer's product (a gated block's) is done with: kind, and for tiles their name and grid."""
    lib = _load()
    out = (ctypes.c_int64 * 8)()
    lib.i8_test_route(ctypes.c_int64(rows), ctypes.c_int64(cols), int(gated), ctypes.c_int64(batch), int(quant), out)
    return _named(out, TILES)


def grad(rows, cols, gated, batch):
    """The same of the gradient with respect to the activations."""
    lib = _load()
    out = (ctypes.c_int64 * 8)()
    lib.i8_test_grad(ctypes.c_int64(rows), ctypes.c_int64(cols), int(gated), ctypes.c_int64(batch), out)
    out[5] = KINDS.index("tiles")
    return _named(out, GRAD_TILES)


def _named(out, names):
    d = dict(zip(("shape", "splits", "steps_per_split", "across", "tok_tiles", "kind", "inside", "ws_bytes"), out))
    d["kind"] = KINDS[d["kind"]]
    d["shape"] = names[d["shape"]] if d["kind"] == "tiles" else None
    d["inside"] = bool(d["inside"])
    return d


def shapes(of_gradient):
    """How many tile shapes the header's table has."""
    return _load().i8_test_shapes(int(of_gradient))


# stages of K in LDS and shares of K of each tile shape: where a kernel's loop turns
RING = {"Large": (2, 1), "Wide": (2, 1), "Middle": (3, 1), "Half": (3, 1), "Small": (3, 2), "Slim": (3, 2), "Least": (3, 2)}
GRAD_RING = {"Large": (3, 1), "Half": (2, 1), "Small": (2, 2), "Deep": (3, 2)}


def _loop(steps, plan, ring):
    """{(steps left behind the loop's whole turns, whether it turns twice)} of a plan's parts."""
    stages, shares = ring
    found = set()
    for part in range(plan["splits"]):
        n = min(steps - part * plan["steps_per_split"], plan["steps_per_split"])
        n = -(-n // shares)
        found.add((n % stages, n >= 2 * stages))
    return found


def product_features(batch, rows, cols, gated):
    """What of the product's kernels these sizes run, one tuple each; the batch and the last step are ragged."""
    p = route(rows, cols, gated, batch)
    if p["kind"] != "tiles":
        return {(p["kind"], gated, p["inside"], rows % 8 == 0)}
    name, where = p["shape"], (p["splits"] > 1, p["tok_tiles"] > 1)
    f = {(name, gated, "grid", *where, rows % 8 == 0)}
    return f | {(name, gated, "loop", *turn) for turn in _loop(-(-cols // 128), p, RING[name]) if turn[1]}


def grad_features(batch, rows, cols, gated):
    p = grad(rows, cols, gated, batch)
    name, per = p["shape"], -(-rows // 64)
    f = {(name, gated, "grid", p["splits"] > 1, p["tok_tiles"] > 1, p["across"] > 1)}
    f |= {(name, gated, "loop", *turn) for turn in _loop(per * (2 if gated else 1), p, GRAD_RING[name]) if turn[1]}
    if gated and p["splits"] > 1 and per % p["steps_per_split"]:
        f.add((name, "both matrices in a part"))
    part = 64 * per
    terms = "any" if rows % 8 or part > 32768 else next(n for n in (2048, 4096, 8192, 16384, 32768) if part <= n)
    return f | {("terms", gated, terms)}
