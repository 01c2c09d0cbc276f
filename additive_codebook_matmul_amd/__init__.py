"""Quantized linear layers on MI355X (gfx950): additive multi-codebook (AQLM) and
microscaled 4-bit (MXFP4).

The compute path is the HIP library libaqlm_mi355x.so (C ABI in
include/aqlm.h and include/aqlm_mx.h); `AqlmLayer` and `MxLayer` are its thin
torch-facing bindings. Importing the package does not load the library; the
first call does, and fails loudly if it has not been built.
"""
from ._lib import (AqlmError, AqlmLayer, gemv_batched, library_path, load_library,  # noqa: F401
                   status_string)
from .mx import MxLayer, mx_dequant, mx_gemv_batched, mx_quantize  # noqa: F401

__all__ = ["AqlmLayer", "AqlmError", "gemv_batched", "load_library", "library_path",
           "status_string", "MxLayer", "mx_quantize", "mx_dequant", "mx_gemv_batched"]
