"""The attention side of a decoder layer: rotary positions, a paged cache of
keys and values, attention of new tokens over it, and the upkeep of its pages.

A thin binding like the package's own: arguments are checked and marshalled,
the kernels behind ``include/bqm.h`` compute. What a caller keeps between
calls are three small objects over its own tensors: ``KvCache`` (the pages'
contents), ``KvPages`` (which sequence holds which pages) and ``KvBatch`` (the
new tokens of a step).
"""
import ctypes
import math
from typing import NamedTuple

from . import _call, _dev_tensor, _i32, _i64, _p, _stream, _sz, _torch, library

_DTYPES = ("float32", "float16", "bfloat16")  # in the order of the header's codes


def _code(dtype):
    try:
        return _DTYPES.index(str(dtype).rsplit(".", 1)[1])
    except ValueError:
        raise TypeError("dtype %s: float32, float16 or bfloat16 expected" % dtype) from None


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


def argtypes(L):
    """Declares the entry points of this module on the loaded library."""
    f, d = ctypes.c_float, ctypes.c_double
    L.rope_table.argtypes = [_p, _p, _i64, _i32, d, _p]
    L.rope.argtypes = [_p, _i64, _i64, _p, _i64, _i64, _p, _p, _i64, _i32, _i32, _i64, _i32, _i32,
                       _i32, _i32, _i32, _p]
    L.rope_kv_append.argtypes = [_p, _p, _p, _i64, _p, _p, _p, _p, _p, _i64, _i32, _i32, _i32,
                                 _i32, _p]
    L.paged_attention.argtypes = [_p, _i64, _i64, _p, _p, _p, _i32, f, _i32, _i32, _i32, _p, _sz,
                                  _p]
    L.paged_attention_workspace_bytes.argtypes = [_p, _p, _i32]
    L.kv_extend.argtypes = [_p, _p, _p, _i32, _p, _p, _sz, _p]
    L.kv_fork.argtypes = [_p, _p, _p, _p, _i32, _i32, _p, _p, _p, _sz, _p]
    L.kv_free.argtypes = [_p, _p, _p, _i32, _p]
    L.kv_compact.argtypes = [_p, _p, _i32, _p, _p, _p]
    L.kv_copy_pages.argtypes = [_p, _p, _i64, _p]
    L.kv_pages_workspace_bytes.argtypes = [_p]
    for name in ("rope_table", "rope", "rope_kv_append", "paged_attention", "kv_extend", "kv_fork",
                 "kv_free", "kv_compact", "kv_copy_pages"):
        getattr(L, name).restype = ctypes.c_int
    L.paged_attention_workspace_bytes.restype = _sz
    L.kv_pages_workspace_bytes.restype = _sz


def _gpu(t, name, dtype, dims, device=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a GPU tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.dim() != dims:
        raise ValueError("%s has %d dimensions, expected %d" % (name, t.dim(), dims))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    return t


def _scratch(need, device, stream):
    """A workspace of this call alone; on a stream other than the current one
    the allocator is told, so that it hands the memory on only after the call."""
    torch = _torch()
    t = torch.empty(need, dtype=torch.uint8, device=device)
    if stream is not None:
        t.record_stream(stream)
    return t


def _ints(t, name, n, device):
    """A contiguous int32 vector of n entries."""
    t = _gpu(t, name, _torch().int32, 1, device)
    if t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be a contiguous vector of %d" % (name, n))
    return t.data_ptr()


class KvCache:
    """Keys and values in pages: two tensors [n_pages, page_size, n_heads,
    head_dim], or with the layers of a model before the pages, float16 or
    bfloat16, of the same strides; any order of pages, tokens and heads in
    memory, a head's values contiguous."""

    def __init__(self, k, v):
        torch = _torch()
        _gpu(k, "k", None, k.dim())
        _gpu(v, "v", k.dtype, k.dim(), k.device)
        if k.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("k has dtype %s, expected float16 or bfloat16" % k.dtype)
        if k.dim() not in (4, 5):
            raise ValueError("k has %d dimensions, expected 4 or 5" % k.dim())
        if k.shape != v.shape or k.stride() != v.stride():
            raise ValueError("k and v differ in shape or strides")
        if k.shape[-1] > 1 and k.stride(-1) != 1:
            raise ValueError("the values of a head must be contiguous")
        self.k, self.v, self.device, self.dtype = k, v, k.device, k.dtype
        self.n_layers = k.shape[0] if k.dim() == 5 else 1
        self.n_pages, self.page_size, self.n_heads, self.head_dim = k.shape[-4:]
        strides = k.stride() if k.dim() == 5 else (0,) + k.stride()
        self.struct = _CacheStruct(k.data_ptr(), v.data_ptr(), strides[0], strides[1], strides[2],
                                   strides[3], self.n_layers, self.n_pages, self.page_size,
                                   self.n_heads, self.head_dim, _code(k.dtype))

    def layer(self, i):
        """The cache of layer i alone (the one attention and the append use)."""
        return KvCache(self.k[i], self.v[i]) if self.k.dim() == 5 else self


class KvBatch:
    """The new tokens of a step: table int32 [n_seqs, max_pages], kv_lens int32
    [n_seqs] (the new tokens counted), q_starts int32 [n_seqs + 1]. max_q and
    max_kv bound the sequences' new tokens and tokens on the host (by default
    whatever the arrays could hold; closer bounds give better launches)."""

    def __init__(self, table, kv_lens, q_starts, max_q=None, max_kv=None):
        torch = _torch()
        _gpu(table, "table", torch.int32, 2)
        n, width = table.shape
        if width > 1 and table.stride(1) != 1:
            raise ValueError("the table's rows must be contiguous")
        self.table, self.kv_lens, self.q_starts, self.device = table, kv_lens, q_starts, table.device
        self.n_seqs, self.max_pages = n, width
        self.max_q, self.max_kv = max_q, max_kv
        self._args = (table.data_ptr(), _ints(kv_lens, "kv_lens", n, table.device),
                      _ints(q_starts, "q_starts", n + 1, table.device), table.stride(0))

    def struct(self, total_q, page_size):
        max_q = total_q if self.max_q is None else self.max_q
        max_kv = min(self.max_pages * page_size, 2 ** 30) if self.max_kv is None else self.max_kv
        return _BatchStruct(*self._args, total_q, self.n_seqs, self.max_pages, max_q, max_kv)


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
    torch = _torch()
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
    torch = _torch()
    _gpu(inv_freq, "inv_freq", torch.float64, 1)
    n = inv_freq.shape[0]
    if out is None:
        out = torch.empty((n_pos, n, 2), dtype=torch.float32, device=inv_freq.device)
    _call("rope_table", _dev_tensor(inv_freq, "inv_freq", (torch.float64,), n * 8),
          _dev_tensor(out, "out", (torch.float32,), n_pos * n * 8, inv_freq.device),
          n_pos, n, scale, _stream(stream, inv_freq.device))
    return out


def _angles(table, device):
    t = _gpu(table, "table", _torch().float32, 3, device)
    if t.shape[2] != 2 or not t.is_contiguous():
        raise ValueError("table must be contiguous [n_pos, n_freq, 2]")
    return t.data_ptr(), t.shape[0], t.shape[1]


def _heads(t, name, dtype=None, device=None):
    _gpu(t, name, dtype, 3, device)
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError("the values of a head of %s must be contiguous" % name)
    return t


def rope(x, table, positions, interleaved=False, inverse=False, out=None, out_dtype=None,
         stream=None):
    """x [T, n_heads, head_dim] (any strides, values contiguous) turned by the
    angles of table (``rope_table``) at positions int32 [T]; ``inverse`` turns
    back (the gradient). out may be x itself."""
    torch = _torch()
    _heads(x, "x")
    T, H, D = x.shape
    if out is None:
        out = torch.empty((T, H, D), dtype=out_dtype or x.dtype, device=x.device)
    elif _heads(out, "out", out_dtype, x.device).shape != x.shape:
        raise ValueError("out has shape %s, expected %s" % (tuple(out.shape), tuple(x.shape)))
    pt, n_pos, n_freq = _angles(table, x.device)
    pp = _ints(positions, "positions", T, x.device)
    if T == 0:
        return out
    _call("rope", x.data_ptr(), x.stride(0), x.stride(1), out.data_ptr(), out.stride(0),
          out.stride(1), pp, pt, T, H, D, n_pos, n_freq, int(interleaved), int(inverse),
          _code(x.dtype), _code(out.dtype), _stream(stream, x.device))
    return out


def rope_kv_append(q, k, v, cache, batch, table, positions=None, interleaved=False, q_out=None,
                   stream=None):
    """Turns q [total_q, n_q_heads, head_dim] into q_out (of the cache's type)
    and k [total_q, n_heads, head_dim] into the cache, and stores v there, at the
    new tokens' places. q, k and v may be slices of one product's rows (one
    stride between rows, heads contiguous); q may be None."""
    torch = _torch()
    _heads(k, "k", None, cache.device)
    _heads(v, "v", k.dtype, cache.device)
    T, H, D = k.shape
    if H != cache.n_heads or D != cache.head_dim or v.shape != k.shape:
        raise ValueError("k and v must be [total_q, %d, %d]" % (cache.n_heads, cache.head_dim))
    n_q = 0 if q is None else _heads(q, "q", k.dtype, cache.device).shape[1]
    if q is not None and (q.shape[0] != T or q.shape[2] != D):
        raise ValueError("q must be [%d, n_q_heads, %d]" % (T, D))
    for t in (k, v) if q is None else (q, k, v):
        if (t.shape[1] > 1 and t.stride(1) != D) or (T > 1 and t.stride(0) != k.stride(0)):
            raise ValueError("q, k and v need contiguous heads and the same stride between rows")
    if q is not None:
        if q_out is None:
            q_out = torch.empty((T, n_q, D), dtype=cache.dtype, device=cache.device)
        elif q_out.shape != q.shape or not q_out.is_contiguous():
            raise ValueError("q_out must be contiguous, of q's shape")
        _heads(q_out, "q_out", cache.dtype, cache.device)
    if batch.device != cache.device:
        raise ValueError("the batch is on %s, expected %s" % (batch.device, cache.device))
    pt, n_pos, n_freq = _angles(table, cache.device)
    pp = None if positions is None else _ints(positions, "positions", T, cache.device)
    if T == 0:
        return q_out
    b = batch.struct(T, cache.page_size)
    _call("rope_kv_append", None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(),
          k.stride(0), None if q is None else q_out.data_ptr(), ctypes.byref(cache.struct),
          ctypes.byref(b), pp, pt, n_pos, n_freq, int(interleaved), n_q, _code(k.dtype),
          _stream(stream, cache.device))
    return q_out


def paged_attention_workspace_bytes(cache, batch, n_q_heads, total_q):
    b = batch.struct(total_q, cache.page_size)
    return int(library().paged_attention_workspace_bytes(ctypes.byref(cache.struct),
                                                         ctypes.byref(b), n_q_heads))


def paged_attention(q, cache, batch, scale=None, causal=True, window=0, out=None, out_dtype=None,
                    workspace=None, stream=None):
    """Attention of q [total_q, n_q_heads, head_dim] (the cache's type; strides
    of multiples of 8) over the batch's pages of the cache; scale defaults to
    head_dim ** -0.5, window 0 is none. out is contiguous, of the cache's type
    or float32; rows that see no token are zeros."""
    torch = _torch()
    _heads(q, "q", cache.dtype, cache.device)
    T, H, D = q.shape
    if D != cache.head_dim:
        raise ValueError("q has heads of %d values, the cache of %d" % (D, cache.head_dim))
    if out is None:
        out = torch.empty((T, H, D), dtype=out_dtype or cache.dtype, device=q.device)
    elif _heads(out, "out", out_dtype, q.device).shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous, of q's shape")
    if batch.device != cache.device:
        raise ValueError("the batch is on %s, expected %s" % (batch.device, cache.device))
    if T == 0:
        return out
    b = batch.struct(T, cache.page_size)
    pc, pb = ctypes.byref(cache.struct), ctypes.byref(b)
    need = library().paged_attention_workspace_bytes(pc, pb, H)
    if need and workspace is None:
        workspace = _scratch(need, q.device, stream)
    pw = None if workspace is None else _dev_tensor(workspace, "workspace", (torch.uint8,), need,
                                                    q.device)
    _call("paged_attention", q.data_ptr(), q.stride(0), q.stride(1), pc, pb, out.data_ptr(), H,
          D ** -0.5 if scale is None else scale, int(causal), window, _code(out.dtype), pw,
          0 if workspace is None else workspace.numel(), _stream(stream, q.device))
    return out


def _pages(p, name="pages", like=None):
    torch = _torch()
    t = _gpu(p.table, name + ".table", torch.int32, 2)
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("the table's rows must be contiguous")
    if like is not None and (t.shape != like.table.shape or t.device != like.table.device or
                             p.refs.shape != like.refs.shape):
        raise ValueError("out differs from pages in its sizes or device")
    n, dev = t.shape[0], t.device
    n_pages = _gpu(p.refs, name + ".refs", torch.int32, 1, dev).shape[0]
    return _PagesStruct(t.data_ptr(), _ints(p.lens, name + ".lens", n, dev),
                        _ints(p.refs, name + ".refs", n_pages, dev), t.stride(0), n_pages, n,
                        t.shape[1])


def _pages_out(pages, out):
    """(struct of pages, out, struct of out, device)"""
    torch = _torch()
    a = _pages(pages)
    if out is None:
        out = KvPages(torch.empty(pages.table.shape, dtype=torch.int32, device=pages.table.device),
                      torch.empty_like(pages.lens), torch.empty_like(pages.refs))
    return a, out, _pages(out, "out", pages), pages.table.device


def _pages_workspace(a, workspace, device, stream):
    torch = _torch()
    need = library().kv_pages_workspace_bytes(ctypes.byref(a))
    if workspace is None:
        workspace = _scratch(need, device, stream)
    return _dev_tensor(workspace, "workspace", (torch.uint8,), need, device), workspace.numel()


def kv_extend(pages, n_new, page_size, out=None, workspace=None, stream=None):
    """Room for n_new int32 [n_seqs] more tokens: (pages, short_of), short_of
    int32 [1] on the GPU the count of sequences that got none. out: where the new
    state goes (pages itself: in place)."""
    torch = _torch()
    a, out, b, dev = _pages_out(pages, out)
    short_of = torch.empty(1, dtype=torch.int32, device=dev)
    pw, nw = _pages_workspace(a, workspace, dev, stream)
    _call("kv_extend", ctypes.byref(a), ctypes.byref(b), _ints(n_new, "n_new", a.n_seqs, dev),
          page_size, short_of.data_ptr(), pw, nw, _stream(stream, dev))
    return out, short_of


def kv_fork(pages, parents, children, page_size, out=None, workspace=None, stream=None):
    """Row children[i] becomes a fork of row parents[i] (int32 [n] both): (pages,
    moves, short_of), moves int32 [n, 3] for ``kv_copy_pages``, short_of as for
    ``kv_extend``."""
    torch = _torch()
    a, out, b, dev = _pages_out(pages, out)
    n = parents.shape[0]
    moves = torch.empty((n, 3), dtype=torch.int32, device=dev)
    short_of = torch.empty(1, dtype=torch.int32, device=dev)
    pw, nw = _pages_workspace(a, workspace, dev, stream)
    pm = moves.data_ptr() if n else short_of.data_ptr()  # nothing is written there without forks
    pp, pc = _ints(parents, "parents", n, dev), _ints(children, "children", n, dev)
    _call("kv_fork", ctypes.byref(a), ctypes.byref(b), pp or pm, pc or pm, n, page_size, pm,
          short_of.data_ptr(), pw, nw, _stream(stream, dev))
    return out, moves, short_of


def kv_free(pages, seqs, out=None, stream=None):
    """The rows seqs int32 [n] end and give their pages back."""
    a, out, b, dev = _pages_out(pages, out)
    n = seqs.shape[0]
    _call("kv_free", ctypes.byref(a), ctypes.byref(b),
          _ints(seqs, "seqs", n, dev) or a.lens, n, _stream(stream, dev))
    return out


def kv_compact(pages, page_size, out=None, stream=None):
    """Used pages move into the free ones before them: (pages, moves, page_map),
    moves int32 [n_pages // 2, 3] for ``kv_copy_pages``, page_map int32 [n_pages]
    where each page's tokens are now."""
    torch = _torch()
    a, out, b, dev = _pages_out(pages, out)
    moves = torch.empty((a.n_pages // 2, 3), dtype=torch.int32, device=dev)
    page_map = torch.empty(a.n_pages, dtype=torch.int32, device=dev)
    pm = moves.data_ptr() or page_map.data_ptr()  # one page: no moves are written
    _call("kv_compact", ctypes.byref(a), ctypes.byref(b), page_size, page_map.data_ptr(), pm,
          _stream(stream, dev))
    return out, moves, page_map


def kv_copy_pages(cache, moves, stream=None):
    """Copies moves int32 [n, 3] = (from page, to page, tokens) in every layer."""
    torch = _torch()
    m = _gpu(moves, "moves", torch.int32, 2, cache.device)
    if m.shape[1] != 3 or not m.is_contiguous():
        raise ValueError("moves must be contiguous [n, 3]")
    if m.shape[0]:
        _call("kv_copy_pages", ctypes.byref(cache.struct), m.data_ptr(), m.shape[0],
              _stream(stream, cache.device))
