"""The attention side of a decoder layer: rotary positions, a paged cache of
keys and values, attention of new tokens over it, and the upkeep of its pages.

What a caller keeps between calls are three small objects over its own tensors:
``KvCache`` (the pages' contents), ``KvPages`` (which sequence holds which
pages) and ``KvBatch`` (the new tokens of a step). The functions are those of
the native module ``_attention`` (``binding/attention.cpp``), which checks and
marshals arguments; the kernels behind ``include/bqm.h`` compute.

``stream=`` runs a call there instead of on the current stream, as if it were the
current one: new outputs and workspaces are that stream's memory (outputs also
count as used by the caller's current stream). What a call reads must be ready
on its stream, and not be let go of before the call has run.
"""
import ctypes
import math
from typing import NamedTuple

import torch

from . import BqmError, _i32, _i64, _p, library

library()  # the C library that _attention links to; raises if it is not built
try:
    from . import _attention
except ImportError as e:
    raise RuntimeError("bit_quantized_mat_amd._attention is not built; run "
                       "bit_quantized_mat_amd.build.build() (or __graft_entry__.build()) first") from e

from ._attention import (KvBatch, KvCache, kv_compact, kv_copy_pages, kv_extend, kv_fork,  # noqa: E402
                         kv_free, paged_attention, paged_attention_workspace_bytes, rope,
                         rope_kv_append, rope_table)

__all__ = ["KvBatch", "KvCache", "KvPages", "kv_compact", "kv_copy_pages", "kv_extend", "kv_fork",
           "kv_free", "paged_attention", "paged_attention_workspace_bytes", "rope", "rope_inv_freq",
           "rope_kv_append", "rope_table"]


class _CacheStruct(ctypes.Structure):
    """bqm_kv_cache, for callers of the C ABI by way of ctypes."""
    _fields_ = [("k", _p), ("v", _p), ("layer_stride", _i64), ("page_stride", _i64),
                ("token_stride", _i64), ("head_stride", _i64), ("n_layers", _i64),
                ("n_pages", _i64), ("page_size", _i32), ("n_heads", _i32), ("head_dim", _i32),
                ("dtype", _i32)]


class _BatchStruct(ctypes.Structure):
    """bqm_kv_batch."""
    _fields_ = [("table", _p), ("kv_lens", _p), ("q_starts", _p), ("table_stride", _i64),
                ("total_q", _i64), ("n_seqs", _i32), ("max_pages", _i32), ("max_q", _i32),
                ("max_kv", _i32)]


class _PagesStruct(ctypes.Structure):
    """bqm_kv_pages."""
    _fields_ = [("table", _p), ("lens", _p), ("refs", _p), ("table_stride", _i64),
                ("n_pages", _i64), ("n_seqs", _i32), ("max_pages", _i32)]


class KvPages(NamedTuple):
    """Which sequences hold which pages: table int32 [n_seqs, max_pages] (-1
    behind each row's end), lens int32 [n_seqs], refs int32 [n_pages]."""
    table: torch.Tensor
    lens: torch.Tensor
    refs: torch.Tensor


_attention.set_python(BqmError, KvPages, torch._C._cuda_getCurrentRawStream)


def rope_inv_freq(n_rot, base=10000.0, factor=1.0, original=None, low=1.0, high=4.0, device="cuda"):
    """The frequencies base**(-2i / n_rot) as fp64 [n_rot / 2] for ``rope_table``,
    scaled for contexts ``factor`` times as long as the trained one: without
    ``original`` all are divided by factor (positions interpolated); with it (the
    trained length) a frequency that turns at least ``high`` times in it stays, one
    that turns at most ``low`` times is divided, and those between are mixed by
    where their turns lie."""
    if n_rot < 2 or n_rot % 2:
        raise ValueError("n_rot must be even and at least 2")
    f = float(base) ** (-torch.arange(0, n_rot, 2, dtype=torch.float64) / n_rot)
    if original is None:
        f = f / factor
    else:
        if not high > low:
            raise ValueError("high must be above low")
        turns = original * f / (2.0 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    return f.to(device)
