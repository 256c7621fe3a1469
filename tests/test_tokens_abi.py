"""CPU checks of the token side's C ABI: bad arguments return before any device
work (pointers are never dereferenced here)."""
import ctypes

import bit_quantized_mat_amd as bqm
from bit_quantized_mat_amd.tokens import _Q4Struct

P = ctypes.c_void_p
GOOD, ODD, FAR = 0x10000, 0x10002, 0x20000
NULL, SHAPE, ALIGN, WORKSPACE, DEVICE = -1, -2, -3, -4, -6
INF, NAN = float("inf"), float("nan")


def call(fn, names, base, **kw):
    args = list(base)
    for k, v in kw.items():
        args[names.index(k)] = v
    return getattr(bqm.library(), fn)(*args)


NORM = ["x", "add", "gain", "sum", "y", "a", "T", "K", "eps", "dtype", "add_dtype", "y_dtype", "stream"]


def norm(**kw):
    base = [P(GOOD), P(FAR), P(GOOD), P(0x30000), P(0x40000), P(0x50000), 3, 64, 1e-6, 2, 0, 1, None]
    return call("rms_norm", NORM, base, **kw)


def test_norm_rejects():
    assert norm() == DEVICE                                    # everything is in order but the device
    assert norm(add=None, sum=None, gain=None) == DEVICE and norm(y=None) == DEVICE and norm(a=None) == DEVICE
    assert norm(sum=P(GOOD)) == DEVICE                          # in place
    assert norm(sum=P(FAR), add_dtype=2) == DEVICE              # over the addend, of the same type
    assert norm(add=None, sum=None, add_dtype=9) == DEVICE and norm(y=None, y_dtype=9) == DEVICE
    assert norm(x=None) == NULL and norm(y=None, a=None) == NULL and norm(sum=None) == NULL
    for kw in (dict(T=-1), dict(T=(1 << 23) + 1), dict(K=0), dict(K=16), dict(K=48), dict(K=65568), dict(K=-32),
               dict(eps=-1e-6), dict(eps=INF), dict(eps=NAN), dict(dtype=3), dict(add_dtype=-1), dict(y_dtype=4),
               dict(sum=P(FAR), add_dtype=0)):
        assert norm(**kw) == SHAPE, kw
    for kw in (dict(x=P(GOOD + 8)), dict(add=P(GOOD + 4)), dict(gain=P(GOOD + 4)), dict(sum=P(GOOD + 8)),
               dict(y=P(GOOD + 8)), dict(a=P(ODD))):
        assert norm(**kw) == ALIGN, kw


def matrix(**kw):
    return ctypes.byref(_Q4Struct(**dict(dict(codes=GOOD, scales=GOOD, zeros=None, N=5, K=256, group=64), **kw)))


MATRIX_BAD = [
    (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(group=0), SHAPE), (dict(group=16), SHAPE),
    (dict(group=256), SHAPE), (dict(group=96), SHAPE), (dict(N=0), SHAPE), (dict(N=1 << 31), SHAPE), (dict(K=0), SHAPE),
    (dict(K=-64), SHAPE), (dict(K=32), SHAPE), (dict(K=288), SHAPE), (dict(K=(1 << 20) + 64), SHAPE),
    (dict(codes=GOOD + 8), ALIGN), (dict(scales=ODD), ALIGN),
]


def test_q4_rejects():
    lib = bqm.library()
    quantize = lambda m=matrix(), x=P(GOOD), dtype=0: lib.q4_quantize(x, m, dtype, None)  # noqa: E731
    mm = lambda m=matrix(), a=P(GOOD), y=P(FAR), T=3: lib.mm_q4(m, a, y, T, P(0x100000), 1 << 40, None)  # noqa: E731
    rows = lambda m=matrix(), r=P(GOOD), o=P(FAR), n=3, f=1.0, t=0: lib.q4_dequantize(m, r, o, n, f, t, None)  # noqa: E731
    for fn in (quantize, mm, rows):
        assert fn() == DEVICE and fn(matrix(zeros=GOOD + 1)) == DEVICE and fn(None) == NULL
        assert fn(matrix(K=1 << 20, group=128)) == DEVICE and fn(matrix(N=(1 << 31) - 1)) == DEVICE
        for kw, rc in MATRIX_BAD:
            assert fn(matrix(**kw)) == rc, kw
    assert quantize(x=None) == NULL and quantize(x=P(GOOD + 8)) == ALIGN and quantize(dtype=3) == SHAPE
    assert mm(a=None) == NULL and mm(y=None) == NULL and mm(a=P(ODD)) == ALIGN and mm(y=P(ODD)) == ALIGN
    assert mm(T=0) == SHAPE and mm(T=65537) == SHAPE and mm(T=65536) == DEVICE
    assert rows(o=None) == NULL and rows(r=P(ODD)) == ALIGN and rows(o=P(FAR + 8)) == ALIGN
    assert rows(n=-1) == SHAPE and rows(n=1 << 31) == SHAPE and rows(t=3) == SHAPE
    assert rows(r=None, n=6) == SHAPE and rows(r=None, n=5) == DEVICE and rows(n=0) == DEVICE


def test_mm_q4_workspace():
    lib = bqm.library()
    for T in (1, 8, 9, 33, 8193, 65536):
        m = matrix(K=4096)
        need = lib.mm_q4_workspace_bytes(m, T)
        if need:
            assert lib.mm_q4(m, P(GOOD), P(FAR), T, None, 1 << 40, None) == WORKSPACE
            assert lib.mm_q4(m, P(GOOD), P(FAR), T, P(0x100000), need - 1, None) == WORKSPACE
            assert lib.mm_q4(m, P(GOOD), P(FAR), T, P(0x100010), need, None) == ALIGN
        assert lib.mm_q4(m, P(GOOD), P(FAR), T, P(0x100000), need, None) == DEVICE
    for m, T in ((None, 9), (matrix(K=288), 9), (matrix(), 0), (matrix(), 65537)):
        assert lib.mm_q4_workspace_bytes(m, T) == 0


SAMPLE = ["logits", "stride", "heat", "k", "p", "least", "u", "tokens", "logprobs", "T", "V", "dtype", "ws",
          "ws_bytes", "stream"]


def sample(**kw):
    base = [P(GOOD), 100, None, None, None, None, P(GOOD), P(FAR), None, 3, 100, 0, P(0x100000), 1 << 40, None]
    return call("sample", SAMPLE, base, **kw)


def test_sample_rejects():
    assert sample() == DEVICE and sample(T=1, stride=0) == DEVICE and sample(V=(1 << 20) - 1, stride=1 << 20) == DEVICE
    assert sample(heat=P(GOOD), k=P(GOOD), p=P(GOOD), least=P(GOOD), logprobs=P(FAR)) == DEVICE
    for k in ("logits", "u", "tokens"):
        assert sample(**{k: None}) == NULL
    for kw in (dict(T=-1), dict(T=65536), dict(V=0), dict(V=1 << 20, stride=1 << 21), dict(dtype=3), dict(stride=99),
               dict(stride=1 << 40)):
        assert sample(**kw) == SHAPE, kw
    for kw in (dict(logits=P(ODD)), dict(logits=P(GOOD + 1), dtype=1), dict(heat=P(ODD)), dict(k=P(ODD)),
               dict(p=P(ODD)), dict(least=P(ODD)), dict(u=P(ODD)), dict(tokens=P(ODD)), dict(logprobs=P(ODD))):
        assert sample(**kw) == ALIGN, kw
    assert sample(logits=P(ODD), dtype=1) == DEVICE


def test_sample_workspace():
    lib = bqm.library()
    for T, V in ((1, 1), (1, 131072), (64, 100003), (65535, (1 << 20) - 1)):
        need = lib.sample_workspace_bytes(T, V)
        assert need % 256 == 0 and need == bqm.sample_workspace_bytes(T, V)
        if need:
            assert sample(T=T, V=V, stride=1 << 20, ws=None) == WORKSPACE
            assert sample(T=T, V=V, stride=1 << 20, ws_bytes=need - 1) == WORKSPACE
            assert sample(T=T, V=V, stride=1 << 20, ws=P(0x100010)) == ALIGN
        assert sample(T=T, V=V, stride=1 << 20, ws_bytes=need) == DEVICE
    for T, V in ((-1, 5), (65536, 5), (4, 0), (4, 1 << 20)):
        assert lib.sample_workspace_bytes(T, V) == 0
