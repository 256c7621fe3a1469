"""CPU checks of the attention side's C ABI: bad arguments return before any
device work (pointers are never dereferenced here)."""
import ctypes

import pytest

import bit_quantized_mat_amd as bqm
from bit_quantized_mat_amd.attention import _BatchStruct, _CacheStruct, _PagesStruct

P = ctypes.c_void_p
GOOD, ODD, FAR = 0x10000, 0x10002, 0x20000
NULL, SHAPE, ALIGN, WORKSPACE, DEVICE = -1, -2, -3, -4, -6


def _struct(cls, base, kw):
    return ctypes.byref(cls(**dict(base, **kw)))


def cache(**kw):
    return _struct(_CacheStruct, dict(k=GOOD, v=GOOD, layer_stride=0, page_stride=16 * 2 * 64,
                                      token_stride=2 * 64, head_stride=64, n_layers=1, n_pages=10,
                                      page_size=16, n_heads=2, head_dim=64, dtype=1), kw)


def batch(**kw):
    return _struct(_BatchStruct, dict(table=GOOD, kv_lens=GOOD, q_starts=GOOD, table_stride=4,
                                      total_q=3, n_seqs=2, max_pages=4, max_q=3, max_kv=64), kw)


def pages(**kw):
    return _struct(_PagesStruct, dict(table=GOOD, lens=GOOD, refs=GOOD, table_stride=4, n_pages=9,
                                      n_seqs=2, max_pages=4), kw)


def call(fn, names, base, **kw):
    args = list(base)
    for k, v in kw.items():
        args[names.index(k)] = v
    return getattr(bqm.library(), fn)(*args)


CACHE_BAD = [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(n_pages=0), SHAPE), (dict(page_size=0), SHAPE),
    (dict(page_size=65537), SHAPE), (dict(n_heads=0), SHAPE), (dict(head_dim=60), SHAPE),
    (dict(head_dim=264), SHAPE), (dict(head_dim=0), SHAPE), (dict(dtype=0), SHAPE), (dict(dtype=3), SHAPE),
    (dict(page_stride=-8), SHAPE), (dict(n_layers=0), SHAPE),
    (dict(page_stride=1 << 33), SHAPE),                       # one layer past 2^35 elements
    (dict(token_stride=132), ALIGN), (dict(head_stride=4), ALIGN), (dict(k=GOOD + 8), ALIGN),
    (dict(v=ODD), ALIGN),
]
BATCH_BAD = [
    (dict(table=None), NULL), (dict(kv_lens=None), NULL), (dict(q_starts=None), NULL),
    (dict(n_seqs=0), SHAPE), (dict(n_seqs=65536), SHAPE), (dict(max_pages=0), SHAPE),
    (dict(total_q=-1), SHAPE), (dict(total_q=(1 << 23) + 1), SHAPE), (dict(max_q=-1), SHAPE),
    (dict(max_kv=-1), SHAPE), (dict(table_stride=-1), SHAPE), (dict(table=ODD), ALIGN),
    (dict(kv_lens=ODD), ALIGN), (dict(q_starts=ODD), ALIGN),
]

ATTN = ["q", "q_token", "q_head", "cache", "batch", "out", "heads", "scale", "causal", "window",
        "out_dtype", "ws", "ws_bytes", "stream"]


def attn(**kw):
    base = [P(GOOD), 4 * 64, 64, cache(), batch(), P(FAR), 4, 0.125, 1, 0, 1, P(0x100000), 1 << 40, None]
    return call("paged_attention", ATTN, base, **kw)


def test_attention_rejects():
    assert attn() == DEVICE                                   # everything is in order but the device
    assert attn(out_dtype=0) == DEVICE
    for kw, rc in CACHE_BAD:
        assert attn(cache=cache(**kw)) == rc, kw
    for kw, rc in BATCH_BAD:
        assert attn(batch=batch(**kw)) == rc, kw
    assert attn(cache=None) == NULL and attn(batch=None) == NULL
    assert attn(q=None) == NULL and attn(out=None) == NULL
    assert attn(heads=0) == SHAPE and attn(heads=3) == SHAPE and attn(heads=-2) == SHAPE
    assert attn(heads=65536) == SHAPE
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert attn(scale=scale) == SHAPE
    assert attn(window=-1) == SHAPE and attn(out_dtype=2) == SHAPE and attn(out_dtype=7) == SHAPE
    assert attn(q_token=-8) == SHAPE and attn(q_head=-8) == SHAPE
    assert attn(q_token=100) == ALIGN and attn(q=P(ODD)) == ALIGN and attn(out=P(FAR + 8)) == ALIGN
    assert attn(ws=P(0x100010)) == ALIGN


def test_attention_workspace():
    # the size is a function of the sizes alone, and a call with less is refused
    lib = bqm.library()
    c = cache(n_pages=1 << 16, page_size=64)
    b = batch(n_seqs=1, total_q=1, max_q=1, max_kv=1 << 20, max_pages=1 << 14)
    need = lib.paged_attention_workspace_bytes(c, b, 8)
    assert need % 256 == 0
    if need:
        assert attn(cache=c, batch=b, heads=8, ws=None) == WORKSPACE
        assert attn(cache=c, batch=b, heads=8, ws_bytes=need - 1) == WORKSPACE
    assert attn(cache=c, batch=b, heads=8, ws_bytes=need) == DEVICE
    assert lib.paged_attention_workspace_bytes(None, b, 8) == 0
    assert lib.paged_attention_workspace_bytes(c, None, 8) == 0
    assert lib.paged_attention_workspace_bytes(c, b, 7) == 0


ROPE = ["x", "xt", "xh", "y", "yt", "yh", "pos", "table", "T", "H", "D", "n_pos", "n_freq", "inter",
        "inverse", "in_dtype", "out_dtype", "stream"]


def rope(**kw):
    base = [P(GOOD), 256, 64, P(FAR), 256, 64, P(GOOD), P(GOOD), 5, 4, 64, 100, 32, 0, 0, 1, 1, None]
    return call("rope", ROPE, base, **kw)


def test_rope_rejects():
    assert rope() == DEVICE and rope(x=P(ODD), xt=257) == DEVICE   # any element alignment
    assert rope(y=P(GOOD)) == DEVICE                               # in place
    for k in ("x", "y", "pos", "table"):
        assert rope(**{k: None}) == NULL
    for kw in (dict(T=-1), dict(T=(1 << 23) + 1), dict(H=0), dict(D=1), dict(D=1025), dict(n_freq=0),
               dict(n_freq=33), dict(n_pos=0), dict(n_pos=1 << 31), dict(in_dtype=3), dict(out_dtype=-1),
               dict(xt=-1), dict(yh=-1), dict(H=1 << 20, D=64),
               dict(y=P(GOOD), yt=300), dict(y=P(GOOD), out_dtype=2)):
        assert rope(**kw) == SHAPE, kw
    assert rope(x=P(GOOD + 1)) == ALIGN and rope(y=P(FAR + 2), out_dtype=0) == ALIGN
    assert rope(pos=P(ODD)) == ALIGN and rope(table=P(GOOD + 4)) == ALIGN


@pytest.mark.parametrize("args,expect", [
    ((None, P(GOOD), 4, 8, 1.0, None), NULL), ((P(GOOD), None, 4, 8, 1.0, None), NULL),
    ((P(GOOD), P(GOOD), 0, 8, 1.0, None), SHAPE), ((P(GOOD), P(GOOD), 1 << 31, 8, 1.0, None), SHAPE),
    ((P(GOOD), P(GOOD), 4, 0, 1.0, None), SHAPE), ((P(GOOD), P(GOOD), 4, 513, 1.0, None), SHAPE),
    ((P(GOOD + 4), P(GOOD), 4, 8, 1.0, None), ALIGN), ((P(GOOD), P(GOOD + 4), 4, 8, 1.0, None), ALIGN),
])
def test_rope_table_rejects(args, expect):
    assert bqm.library().rope_table(*args) == expect


APPEND = ["q", "k", "v", "stride", "q_out", "cache", "batch", "pos", "table", "n_pos", "n_freq", "inter",
          "heads", "in_dtype", "stream"]


def append(**kw):
    base = [P(GOOD), P(GOOD), P(GOOD), 8 * 64, P(FAR), cache(), batch(), None, P(GOOD), 100, 32, 0, 4, 0, None]
    return call("rope_kv_append", APPEND, base, **kw)


def test_append_rejects():
    assert append() == DEVICE and append(q=None, q_out=None, heads=0) == DEVICE
    for kw, rc in CACHE_BAD:
        assert append(cache=cache(**kw)) == rc, kw
    for kw, rc in BATCH_BAD:
        assert append(batch=batch(**kw)) == rc, kw
    for k in ("q", "k", "v", "q_out", "table", "cache", "batch"):
        assert append(**{k: None}) == NULL, k
    for kw in (dict(heads=-1), dict(n_freq=33), dict(n_freq=0), dict(n_pos=0), dict(stride=-1),
               dict(in_dtype=3), dict(heads=1 << 18)):
        assert append(**kw) == SHAPE, kw
    for kw in (dict(k=P(ODD)), dict(q=P(ODD)), dict(q_out=P(FAR + 8)), dict(table=P(GOOD + 4)),
               dict(pos=P(ODD))):
        assert append(**kw) == ALIGN, kw


PAGES_BAD = [
    (dict(table=None), NULL), (dict(lens=None), NULL), (dict(refs=None), NULL), (dict(n_pages=0), SHAPE),
    (dict(n_pages=(1 << 30) + 1), SHAPE), (dict(n_seqs=0), SHAPE), (dict(n_seqs=65536), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(table_stride=3), SHAPE), (dict(refs=ODD), ALIGN),
    (dict(table=ODD), ALIGN),
]
WS, BIG = P(0x100000), 1 << 40
UPKEEP = {
    "kv_extend": (["in", "out", "n_new", "ps", "short", "ws", "bytes", "stream"],
                  [None, None, P(GOOD), 16, P(GOOD), WS, BIG, None]),
    "kv_fork": (["in", "out", "parents", "children", "n", "ps", "moves", "short", "ws", "bytes", "stream"],
                [None, None, P(GOOD), P(GOOD), 2, 16, P(GOOD), P(GOOD), WS, BIG, None]),
    "kv_free": (["in", "out", "seqs", "n", "stream"], [None, None, P(GOOD), 2, None]),
    "kv_compact": (["in", "out", "ps", "page_map", "moves", "stream"],
                   [None, None, 16, P(GOOD), P(GOOD), None]),
}


@pytest.mark.parametrize("fn", sorted(UPKEEP))
def test_upkeep_rejects(fn):
    names, base = UPKEEP[fn]

    def up(**kw):
        return call(fn, names, base, **dict({"in": pages(), "out": pages()}, **kw))

    assert up() == DEVICE
    for kw, rc in PAGES_BAD:
        assert up(**{"in": pages(**kw)}) == rc, kw
        assert up(out=pages(**kw)) == rc, kw
    for kw in (dict(n_pages=8), dict(n_seqs=3), dict(max_pages=3), dict(table_stride=5)):
        assert up(out=pages(**kw)) == SHAPE, kw       # other sizes, or in place at another stride
    assert up(**{"in": None}) == NULL and up(out=None) == NULL
    for k in set(names) & {"n_new", "short", "parents", "children", "moves", "seqs", "page_map"}:
        assert up(**{k: None}) == NULL, k
        assert up(**{k: P(ODD)}) == ALIGN, k
    if "ps" in names:
        assert up(ps=0) == SHAPE and up(ps=65537) == SHAPE
    if "n" in names:
        assert up(n=-1) == SHAPE and up(n=65536) == SHAPE and up(n=0) == DEVICE
    if fn == "kv_fork":
        assert up(n=3) == SHAPE                        # more forks than rows
    if "ws" in names:
        need = bqm.library().kv_pages_workspace_bytes(pages())
        assert need > 0 and need % 256 == 0
        assert up(ws=None) == WORKSPACE and up(bytes=need - 1) == WORKSPACE and up(bytes=need) == DEVICE
        assert up(ws=P(0x100010)) == ALIGN


def test_copy_rejects():
    lib = bqm.library()
    assert lib.kv_copy_pages(cache(), P(GOOD), 2, None) == DEVICE
    for kw, rc in CACHE_BAD:
        assert lib.kv_copy_pages(cache(**kw), P(GOOD), 2, None) == rc, kw
    assert lib.kv_copy_pages(None, P(GOOD), 2, None) == NULL
    assert lib.kv_copy_pages(cache(), None, 2, None) == NULL
    assert lib.kv_copy_pages(cache(), P(GOOD), -1, None) == SHAPE
    assert lib.kv_copy_pages(cache(), P(ODD), 2, None) == ALIGN
    assert lib.kv_pages_workspace_bytes(None) == 0
    assert lib.kv_pages_workspace_bytes(pages(n_pages=0)) == 0
