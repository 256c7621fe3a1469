"""The attention side of a decoder layer: rotary positions, a paged cache of
keys and values, attention of new tokens over it, and the upkeep of its pages.

A thin binding like the package's own: arguments are checked and marshalled,
the kernels behind ``include/bqm.h`` compute. What a caller keeps between
calls are three small objects over its own tensors: ``KvCache`` (the pages'
contents), ``KvPages`` (which sequence holds which pages) and ``KvBatch`` (the
new tokens of a step).

A decode step's smallest kernels take a few microseconds, so the checks here
are written to cost little: one test a tensor, its message only when it fails.
"""
import ctypes
import math
from typing import NamedTuple

import torch

from . import BqmError, _i32, _i64, _p, library

_CODES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}  # the header's
_raw_stream = torch._C._cuda_getCurrentRawStream


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("layer_stride", _i64), ("page_stride", _i64),
                ("token_stride", _i64), ("head_stride", _i64), ("n_layers", _i64),
                ("n_pages", _i64), ("page_size", _i32), ("n_heads", _i32), ("head_dim", _i32),
                ("dtype", _i32)]


class _BatchStruct(ctypes.Structure):
    _fields_ = [("table", _p), ("kv_lens", _p), ("q_starts", _p), ("table_stride", _i64),
                ("total_q", _i64), ("n_seqs", _i32), ("max_pages", _i32), ("max_q", _i32),
                ("max_kv", _i32)]


class _PagesStruct(ctypes.Structure):
    _fields_ = [("table", _p), ("lens", _p), ("refs", _p), ("table_stride", _i64),
                ("n_pages", _i64), ("n_seqs", _i32), ("max_pages", _i32)]


def _done(fn, status):
    if status:
        raise BqmError(fn, status)


def _code(dtype):
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("dtype %s: float32, float16 or bfloat16 expected" % dtype)
    return code


def _refuse(t, name, dtype, dims, dev):
    """Says what is wrong with an argument."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a GPU tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.dim() != dims:
        raise ValueError("%s has %d dimensions, expected %d" % (name, t.dim(), dims))
    raise ValueError("%s is on GPU %d, expected %d" % (name, t.get_device(), dev))


def _gpu(t, name, dtype, dims, dev=None):
    """Checks t and returns the index of its GPU (dev, if given)."""
    try:
        at = t.get_device()
        if (at == dev if dev is not None else at >= 0) and t.dim() == dims and (
                dtype is None or t.dtype is dtype):
            return at
    except AttributeError:
        pass
    _refuse(t, name, dtype, dims, dev)


def _ints(t, name, n, dev):
    """The address of a contiguous int32 vector of n entries."""
    _gpu(t, name, torch.int32, 1, dev)
    if t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be a contiguous vector of %d" % (name, n))
    return t.data_ptr()


def _heads(t, name, dtype, dev=None):
    """Checks [tokens, heads, values] with contiguous values; (shape, strides)."""
    _gpu(t, name, dtype, 3, dev)
    shape, strides = t.shape, t.stride()
    if strides[2] != 1 and shape[2] > 1:
        raise ValueError("the values of a head of %s must be contiguous" % name)
    return shape, strides


def _on(stream, dev):
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _scratch(workspace, need, like, stream):
    """(address, bytes, the tensor that holds them) of a workspace: the caller's, or
    one of this call alone; on a stream other than the current one the allocator
    is told, so that it hands the memory on only after the call."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
        if stream is not None:
            workspace.record_stream(stream)
        return workspace.data_ptr(), need, workspace
    _gpu(workspace, "workspace", torch.uint8, 1, like.get_device())
    n = workspace.shape[0]
    if n < need or (n > 1 and workspace.stride(0) != 1):
        raise ValueError("workspace must be %d contiguous bytes" % need)
    return workspace.data_ptr(), n, workspace


class KvCache:
    """Keys and values in pages: two tensors [n_pages, page_size, n_heads,
    head_dim], or with the layers of a model before the pages, float16 or
    bfloat16, of the same strides; any order of pages, tokens and heads in
    memory, a head's values contiguous."""

    __slots__ = ("k", "v", "device", "dtype", "dev", "n_pages", "page_size", "n_heads", "head_dim",
                 "struct", "ref")

    def __init__(self, k, v):
        dims = k.dim() if isinstance(k, torch.Tensor) else 4
        self.dev = _gpu(k, "k", None, dims)
        self.dtype = k.dtype
        _gpu(v, "v", self.dtype, dims, self.dev)
        if self.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("k has dtype %s, expected float16 or bfloat16" % self.dtype)
        if dims not in (4, 5):
            raise ValueError("k has %d dimensions, expected 4 or 5" % dims)
        shape, strides = k.shape, k.stride()
        if shape != v.shape or strides != v.stride():
            raise ValueError("k and v differ in shape or strides")
        if strides[-1] != 1 and shape[-1] > 1:
            raise ValueError("the values of a head must be contiguous")
        self.k, self.v, self.device = k, v, k.device
        self.n_pages, self.page_size, self.n_heads, self.head_dim = shape[-4:]
        layers, layer_stride = (shape[0], strides[0]) if dims == 5 else (1, 0)
        self.struct = _CacheStruct(k.data_ptr(), v.data_ptr(), layer_stride, strides[-4],
                                   strides[-3], strides[-2], layers, self.n_pages, self.page_size,
                                   self.n_heads, self.head_dim, _CODES[self.dtype])
        self.ref = ctypes.byref(self.struct)

    def layer(self, i):
        """The cache of layer i alone (the one attention and the append use)."""
        return KvCache(self.k[i], self.v[i]) if self.k.dim() == 5 else self


class KvBatch:
    """The new tokens of a step: table int32 [n_seqs, max_pages], kv_lens int32
    [n_seqs] (the new tokens counted), q_starts int32 [n_seqs + 1]. max_q and
    max_kv bound the sequences' new tokens and tokens on the host (by default
    whatever the arrays could hold; closer bounds give better launches)."""

    __slots__ = ("table", "kv_lens", "q_starts", "dev", "n_seqs", "max_pages", "max_q", "max_kv",
                 "_args")

    def __init__(self, table, kv_lens, q_starts, max_q=None, max_kv=None):
        self.dev = _gpu(table, "table", torch.int32, 2)
        n, width = table.shape
        row, one = table.stride()
        if one != 1 and width > 1:
            raise ValueError("the table's rows must be contiguous")
        self.table, self.kv_lens, self.q_starts = table, kv_lens, q_starts
        self.n_seqs, self.max_pages, self.max_q, self.max_kv = n, width, max_q, max_kv
        self._args = (table.data_ptr(), _ints(kv_lens, "kv_lens", n, self.dev),
                      _ints(q_starts, "q_starts", n + 1, self.dev), row)

    def ref(self, total_q, cache):
        if self.dev != cache.dev:
            raise ValueError("the batch is on GPU %d, expected %d" % (self.dev, cache.dev))
        max_q = total_q if self.max_q is None else self.max_q
        max_kv = self.max_kv
        if max_kv is None:
            max_kv = min(self.max_pages * cache.page_size, 2 ** 30)
        return ctypes.byref(_BatchStruct(*self._args, total_q, self.n_seqs, self.max_pages, max_q,
                                         max_kv))


class KvPages(NamedTuple):
    """Which sequences hold which pages: table int32 [n_seqs, max_pages] (-1
    behind each row's end), lens int32 [n_seqs], refs int32 [n_pages]."""
    table: object
    lens: object
    refs: object


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


def rope_table(inv_freq, n_pos, scale=1.0, out=None, stream=None):
    """(cos, sin) of position * inv_freq times scale: fp32 [n_pos, n_freq, 2]."""
    dev = _gpu(inv_freq, "inv_freq", torch.float64, 1)
    n = inv_freq.shape[0]
    if n > 1 and inv_freq.stride(0) != 1:
        raise ValueError("inv_freq must be contiguous")
    if out is None:
        out = torch.empty((n_pos, n, 2), dtype=torch.float32, device=inv_freq.device)
    p, rows, freqs = _angles(out, dev)
    if rows != n_pos or freqs != n:
        raise ValueError("out must be [%d, %d, 2]" % (n_pos, n))
    _done("rope_table", library().rope_table(inv_freq.data_ptr(), p, n_pos, n, scale,
                                             _on(stream, dev)))
    return out


def _angles(table, dev):
    _gpu(table, "table", torch.float32, 3, dev)
    n_pos, n_freq, two = table.shape
    if two != 2 or not table.is_contiguous():
        raise ValueError("table must be contiguous [n_pos, n_freq, 2]")
    return table.data_ptr(), n_pos, n_freq


def rope(x, table, positions, interleaved=False, inverse=False, out=None, out_dtype=None,
         stream=None):
    """x [T, n_heads, head_dim] (any strides, values contiguous) turned by the
    angles of table (``rope_table``) at positions int32 [T]; ``inverse`` turns
    back (the gradient). out may be x itself."""
    shape, (x_token, x_head, _) = _heads(x, "x", None)
    dev = x.get_device()
    T, H, D = shape
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or x.dtype, device=x.device)
    out_shape, (y_token, y_head, _) = _heads(out, "out", out_dtype, dev)
    if out_shape != shape:
        raise ValueError("out has shape %s, expected %s" % (tuple(out_shape), tuple(shape)))
    pt, n_pos, n_freq = _angles(table, dev)
    pp = _ints(positions, "positions", T, dev)
    if T:
        _done("rope", library().rope(x.data_ptr(), x_token, x_head, out.data_ptr(), y_token, y_head,
                                     pp, pt, T, H, D, n_pos, n_freq, interleaved, inverse,
                                     _code(x.dtype), _code(out.dtype), _on(stream, dev)))
    return out


def rope_kv_append(q, k, v, cache, batch, table, positions=None, interleaved=False, q_out=None,
                   stream=None):
    """Turns q [total_q, n_q_heads, head_dim] into q_out (of the cache's type)
    and k [total_q, n_heads, head_dim] into the cache, and stores v there, at the
    new tokens' places. q, k and v may be slices of one product's rows (one
    stride between rows, heads contiguous); q may be None."""
    dev, D = cache.dev, cache.head_dim
    dtype = k.dtype if isinstance(k, torch.Tensor) else None
    shape, strides = _heads(k, "k", dtype, dev)
    T, H, d = shape
    v_shape, v_strides = _heads(v, "v", dtype, dev)
    if H != cache.n_heads or d != D or v_shape != shape:
        raise ValueError("k and v must be [total_q, %d, %d]" % (cache.n_heads, D))
    same = H == 1 or strides[1] == v_strides[1] == D
    same = same and (T <= 1 or strides[0] == v_strides[0])
    n_q, pq, po = 0, None, None
    if q is not None:
        q_shape, q_strides = _heads(q, "q", dtype, dev)
        n_q = q_shape[1]
        if q_shape[0] != T or q_shape[2] != D:
            raise ValueError("q must be [%d, n_q_heads, %d]" % (T, D))
        same = same and (n_q == 1 or q_strides[1] == D) and (T <= 1 or q_strides[0] == strides[0])
        if q_out is None:
            q_out = torch.empty(q_shape, dtype=cache.dtype, device=cache.device)
        else:
            _gpu(q_out, "q_out", cache.dtype, 3, dev)
            if q_out.shape != q_shape or not q_out.is_contiguous():
                raise ValueError("q_out must be contiguous, of q's shape")
        pq, po = q.data_ptr(), q_out.data_ptr()
    if not same:
        raise ValueError("q, k and v need contiguous heads and the same stride between rows")
    pt, n_pos, n_freq = _angles(table, dev)
    pp = None if positions is None else _ints(positions, "positions", T, dev)
    b = batch.ref(T, cache)
    if T:
        _done("rope_kv_append", library().rope_kv_append(
            pq, k.data_ptr(), v.data_ptr(), strides[0], po, cache.ref, b, pp, pt, n_pos, n_freq,
            interleaved, n_q, _code(dtype), _on(stream, dev)))
    return q_out


def paged_attention_workspace_bytes(cache, batch, n_q_heads, total_q):
    return library().paged_attention_workspace_bytes(cache.ref, batch.ref(total_q, cache),
                                                     n_q_heads)


def paged_attention(q, cache, batch, scale=None, causal=True, window=0, out=None, out_dtype=None,
                    workspace=None, stream=None):
    """Attention of q [total_q, n_q_heads, head_dim] (the cache's type; strides
    of multiples of 8) over the batch's pages of the cache; scale defaults to
    head_dim ** -0.5, window 0 is none. out is contiguous, of the cache's type
    or float32; rows that see no token are zeros."""
    dev, dtype = cache.dev, cache.dtype
    shape, (q_token, q_head, _) = _heads(q, "q", dtype, dev)
    T, H, D = shape
    if D != cache.head_dim:
        raise ValueError("q has heads of %d values, the cache of %d" % (D, cache.head_dim))
    if out is None:
        dtype = out_dtype or dtype
        out = torch.empty(shape, dtype=dtype, device=cache.device)
    else:
        _gpu(out, "out", out_dtype, 3, dev)
        dtype = out.dtype
        if out.shape != shape or not out.is_contiguous():
            raise ValueError("out must be contiguous, of q's shape")
    b = batch.ref(T, cache)
    if T:
        L = library()
        need = L.paged_attention_workspace_bytes(cache.ref, b, H)
        pw, nw, _keep = _scratch(workspace, need, q, stream)
        _done("paged_attention", L.paged_attention(
            q.data_ptr(), q_token, q_head, cache.ref, b, out.data_ptr(), H,
            D ** -0.5 if scale is None else scale, causal, window, _code(dtype), pw, nw,
            _on(stream, dev)))
    return out


def _pages(p, name, dev=None):
    dev = _gpu(p.table, name + ".table", torch.int32, 2, dev)
    n, width = p.table.shape
    row, one = p.table.stride()
    if one != 1 and width > 1:
        raise ValueError("the table's rows must be contiguous")
    _gpu(p.refs, name + ".refs", torch.int32, 1, dev)
    n_pages = p.refs.shape[0]
    return _PagesStruct(p.table.data_ptr(), _ints(p.lens, name + ".lens", n, dev),
                        _ints(p.refs, name + ".refs", n_pages, dev), row, n_pages, n, width), dev


def _pages_out(pages, out):
    """(struct of pages, reference to it, out, reference to its struct, GPU)"""
    a, dev = _pages(pages, "pages")
    ref = ctypes.byref(a)
    if out is pages:
        return a, ref, out, ref, dev
    if out is None:
        table = torch.empty((a.n_seqs, a.max_pages), dtype=torch.int32, device=pages.table.device)
        out = KvPages(table, torch.empty_like(pages.lens), torch.empty_like(pages.refs))
        b = _PagesStruct(table.data_ptr(), out.lens.data_ptr(), out.refs.data_ptr(), a.max_pages,
                         a.n_pages, a.n_seqs, a.max_pages)
    else:
        b, _ = _pages(out, "out", dev)
        if out.table.shape != pages.table.shape or b.n_pages != a.n_pages:
            raise ValueError("out differs from pages in its sizes")
    return a, ref, out, ctypes.byref(b), dev


def kv_extend(pages, n_new, page_size, out=None, workspace=None, stream=None):
    """Room for n_new int32 [n_seqs] more tokens: (pages, short_of), short_of
    int32 [1] on the GPU the count of sequences that got none. out: where the new
    state goes (pages itself: in place)."""
    a, ra, out, rb, dev = _pages_out(pages, out)
    short_of = torch.empty(1, dtype=torch.int32, device=pages.lens.device)
    L = library()
    pw, nw, _keep = _scratch(workspace, L.kv_pages_workspace_bytes(ra), pages.lens, stream)
    _done("kv_extend", L.kv_extend(ra, rb, _ints(n_new, "n_new", a.n_seqs, dev), page_size,
                                   short_of.data_ptr(), pw, nw, _on(stream, dev)))
    return out, short_of


def kv_fork(pages, parents, children, page_size, out=None, workspace=None, stream=None):
    """Row children[i] becomes a fork of row parents[i] (int32 [n] both): (pages,
    moves, short_of), moves int32 [n, 3] for ``kv_copy_pages``, short_of as for
    ``kv_extend``."""
    a, ra, out, rb, dev = _pages_out(pages, out)
    _gpu(parents, "parents", torch.int32, 1, dev)
    n = parents.shape[0]
    moves = torch.empty((n, 3), dtype=torch.int32, device=pages.lens.device)
    short_of = torch.empty(1, dtype=torch.int32, device=pages.lens.device)
    L = library()
    pw, nw, _keep = _scratch(workspace, L.kv_pages_workspace_bytes(ra), pages.lens, stream)
    ps = short_of.data_ptr()  # stands for the addresses of empty arrays
    _done("kv_fork", L.kv_fork(ra, rb, _ints(parents, "parents", n, dev) or ps,
                               _ints(children, "children", n, dev) or ps, n, page_size,
                               moves.data_ptr() or ps, ps, pw, nw, _on(stream, dev)))
    return out, moves, short_of


def kv_free(pages, seqs, out=None, stream=None):
    """The rows seqs int32 [n] end and give their pages back."""
    a, ra, out, rb, dev = _pages_out(pages, out)
    _gpu(seqs, "seqs", torch.int32, 1, dev)
    n = seqs.shape[0]
    _done("kv_free", library().kv_free(ra, rb, _ints(seqs, "seqs", n, dev) or a.lens, n,
                                       _on(stream, dev)))
    return out


def kv_compact(pages, page_size, out=None, stream=None):
    """Used pages move into the free ones before them: (pages, moves, page_map),
    moves int32 [n_pages // 2, 3] for ``kv_copy_pages``, page_map int32 [n_pages]
    where each page's tokens are now."""
    a, ra, out, rb, dev = _pages_out(pages, out)
    moves = torch.empty((a.n_pages // 2, 3), dtype=torch.int32, device=pages.lens.device)
    page_map = torch.empty_like(pages.refs)
    pm = page_map.data_ptr()  # one page: no moves are written
    _done("kv_compact", library().kv_compact(ra, rb, page_size, pm, moves.data_ptr() or pm,
                                             _on(stream, dev)))
    return out, moves, page_map


def kv_copy_pages(cache, moves, stream=None):
    """Copies moves int32 [n, 3] = (from page, to page, tokens) in every layer."""
    _gpu(moves, "moves", torch.int32, 2, cache.dev)
    n, three = moves.shape
    if three != 3 or not moves.is_contiguous():
        raise ValueError("moves must be contiguous [n, 3]")
    if n:
        _done("kv_copy_pages", library().kv_copy_pages(cache.ref, moves.data_ptr(), n,
                                                       _on(stream, cache.dev)))
