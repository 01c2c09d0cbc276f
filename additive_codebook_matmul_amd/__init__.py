"""Quantized linear layers on MI355X (gfx950): additive multi-codebook (AQLM),
microscaled 4-bit (MXFP4) and 8-bit integer (int8, with gated blocks).

The compute path is the HIP library libaqlm_mi355x.so (C ABI in
include/aqlm.h, include/aqlm_mx.h and include/aqlm_i8.h); `AqlmLayer`, `MxLayer`,
`I8Layer` and `I8Gated` are its thin torch-facing bindings. Importing the package
does not load the library; the first call does, and fails loudly if it has not
been built.
"""
from ._lib import (AqlmError, AqlmLayer, gemv_batched, library_path, load_library,  # noqa: F401
                   status_string)
from .i8 import I8Gated, I8Layer, i8_dequant, i8_quantize  # noqa: F401
from .mx import MxLayer, mx_dequant, mx_gemv_batched, mx_quantize  # noqa: F401

__all__ = ["AqlmLayer", "AqlmError", "gemv_batched", "load_library", "library_path",
           "status_string", "MxLayer", "mx_quantize", "mx_dequant", "mx_gemv_batched",
           "I8Layer", "I8Gated", "i8_quantize", "i8_dequant"]
