"""The token side of a decoder: rows of a table kept in 4 bits, the norm in front of
every product, products of 4-bit matrices and the choice of the next token.

The functions are those of the native module ``_tokens`` (``binding/tokens.cpp``),
which checks and marshals arguments; the kernels behind ``include/bqm.h`` compute.
``stream=`` is as in ``attention.py``.
"""
import ctypes

import torch

from . import BqmError, _i32, _i64, _p, library

library()  # the C library that _tokens links to; raises if it is not built
try:
    from . import _tokens
except ImportError as e:
    raise RuntimeError("bit_quantized_mat_amd._tokens is not built; run "
                       "bit_quantized_mat_amd.build.build() (or __graft_entry__.build()) first") from e

from ._tokens import (Q4Matrix, mm_q4, mm_q4_workspace_bytes, q4_dequantize, q4_quantize,  # noqa: E402
                      rms_norm, rms_norm_q8_1, sample)

__all__ = ["Q4Matrix", "mm_q4", "mm_q4_workspace_bytes", "q4_dequantize", "q4_quantize", "rms_norm",
           "rms_norm_q8_1", "sample", "sample_workspace_bytes"]


class _Q4Struct(ctypes.Structure):
    """bqm_q4_matrix, for callers of the C ABI by way of ctypes."""
    _fields_ = [("codes", _p), ("scales", _p), ("zeros", _p), ("N", _i64), ("K", _i64), ("group", _i32)]


_tokens.set_python(BqmError, torch._C._cuda_getCurrentRawStream)


def sample_workspace_bytes(T, V):
    """Bytes of the uint8 tensor that ``sample(..., workspace=)`` takes for up to T rows (0: none)."""
    return int(library().sample_workspace_bytes(T, V))
