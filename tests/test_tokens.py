"""The token side on the GPU against plain forms in 64 bits: the norm, 4-bit matrices,
sampling."""
import math

import numpy as np
import pytest
import torch

import bit_quantized_mat_amd as bqm
import oracle

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
H32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half a step below a type's normal range."""
    return torch.finfo(t).tiny * torch.finfo(t).eps / 2


def randn(*shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


# ---- the norm ---------------------------------------------------------------------------------------------------------

def check_norm(x, gain, add, eps, out_dtype):
    y, s = bqm.rms_norm(x, gain, add=add, eps=eps, out_dtype=out_dtype)
    want_s = x if add is None else (x.float() + add.float()).to(x.dtype)
    assert torch.equal(s, want_s)
    assert y.dtype == out_dtype and y.shape == x.shape
    d = want_s.double()
    want = d / (d.square().mean(-1, keepdim=True) + eps).sqrt() * (1.0 if gain is None else gain.double())
    # r, s * r and its product with gain are rounded to fp32, then all to the output's type
    rel = (1 + H32) ** 3 * (1 + half_step(out_dtype)) - 1 + 2.0 ** -45
    off = (y.double() - want).abs()
    assert bool((off <= rel * want.abs() + tiny(out_dtype) + 3 * tiny(F32)).all()), float((off / want.abs()).max())
    y32, _ = bqm.rms_norm(x, gain, add=add, eps=eps, out_dtype=F32)
    a, s = bqm.rms_norm_q8_1(x, gain, add=add, eps=eps)
    assert torch.equal(s, want_s)
    assert torch.equal(a, bqm.q8_1_quantize(y32))
    assert np.array_equal(a.cpu().numpy(), oracle.q8_1_quantize(y32.cpu().numpy()))


@pytest.mark.parametrize("K", [32, 96, 480, 512, 544, 1024, 1056, 2016, 4096, 5120, 8192, 8224, 16384, 16416, 32768, 65536])
@pytest.mark.parametrize("T", [1, 2, 5, 33])
def test_norm_sizes(T, K):
    check_norm(randn(T, K, seed=K + T, dtype=BF16, scale=3.0), 1.0 + randn(K, seed=1) * 0.1,
               randn(T, K, seed=K - T), 1e-6, F32)


@pytest.mark.parametrize("out", [F32, F16, BF16])
@pytest.mark.parametrize("add", [None, F32, F16, BF16])
@pytest.mark.parametrize("stream", [F32, F16, BF16])
def test_norm_types(stream, add, out):
    for K in (64, 1600, 9216):
        check_norm(randn(7, K, seed=K, dtype=stream, scale=2.0), None if K == 64 else randn(K, seed=2),
                   None if add is None else randn(7, K, seed=3, dtype=add), 1e-5, out)


def test_norm_values():
    # rows of zeros, of tiny and of huge values beside one another: a square that passes fp32's range either way
    x = randn(5, 1024, seed=4)
    x[0] = 0.0
    x[1] *= 1e-30
    x[2] *= 1e30
    x[3, 1:] = 0.0
    check_norm(x, None, None, 1e-6, F32)
    y, _ = bqm.rms_norm(x, eps=0.0)
    assert torch.isnan(y[0]).all() and torch.isfinite(y[1:]).all()
    x[4, 7] = float("inf")
    y, _ = bqm.rms_norm(x)
    assert torch.isnan(y[4, 7]) and (y[4, :7] == 0).all() and torch.isfinite(y[:4]).all()


@pytest.mark.parametrize("where", ["x", "add", "other"])
def test_norm_in_place(where):
    x, add = randn(9, 2080, seed=5, dtype=BF16), randn(9, 2080, seed=6, dtype=BF16)
    want_y, want_s = bqm.rms_norm(x, add=add)
    to = {"x": x, "add": add, "other": torch.full_like(x, float("nan"))}[where]
    out = torch.full_like(x, float("nan"))
    y, s = bqm.rms_norm(x, add=add, sum_out=to, out=out)
    assert s is to or s.data_ptr() == to.data_ptr()
    assert torch.equal(s, want_s) and torch.equal(y, want_y) and y.data_ptr() == out.data_ptr()


def test_norm_without_addend():
    x = randn(3, 64, seed=7)
    y, s = bqm.rms_norm(x)
    assert s.data_ptr() == x.data_ptr()
    copy = torch.empty_like(x)
    y2, s = bqm.rms_norm(x, sum_out=copy)
    assert torch.equal(copy, x) and torch.equal(y, y2)
    y, s = bqm.rms_norm(x[:0])
    assert y.shape == (0, 64) and bqm.rms_norm_q8_1(x[:0])[0].shape == (0, 72)


def test_norm_refuses():
    x, add = randn(4, 64, seed=8), randn(4, 64, seed=9)
    for bad, err in (((x.cpu(),), TypeError), ((x.double(),), TypeError), ((x[:, ::2],), ValueError), ((x[0],), ValueError),
                     ((x, randn(63, seed=1)), ValueError), ((x, randn(64, seed=1, dtype=BF16)), TypeError)):
        for f in (bqm.rms_norm, bqm.rms_norm_q8_1):
            with pytest.raises(err):
                f(*bad)
    for kw, err in ((dict(add=add[:3]), ValueError), (dict(add=add.double()), TypeError), (dict(eps=-1.0), bqm.BqmError),
                    (dict(add=add, sum_out=add.half()), TypeError), (dict(out=x[:2]), ValueError)):
        with pytest.raises(err):
            bqm.rms_norm(x, **kw)
    with pytest.raises(bqm.BqmError):
        bqm.rms_norm(randn(4, 48, seed=1))
    with pytest.raises(bqm.BqmError):
        bqm.rms_norm(randn(4 * 64 + 1, seed=1)[1:].view(4, 64))  # not 16-byte aligned


# ---- 4-bit matrices ----------------------------------------------------------------------------------------------------

def make_matrix(N, K, group, zeros, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand(N, K // group, generator=g, device="cuda") - 0.3) * 0.1).half()
    z = torch.randint(-8, 8, (N, K // group), generator=g, device="cuda", dtype=torch.int8) if zeros else None
    return bqm.Q4Matrix(codes, scales, z)


def steps_of(m):
    """code - zero of every value, fp64 [N, K], from the layout's definition."""
    N, K = m.N, m.K
    out = np.empty((N, K // 32, 32))
    b = m.codes.cpu().numpy().reshape(N, K // 32, 16)
    for i in range(16):
        for half in range(2):
            c = (b[:, :, i] >> (4 * half)) & 15
            out[:, :, i + 16 * half] = c.astype(np.int64) - 16 * (c >= 8)
    out = out.reshape(N, K)
    if m.zeros is not None:
        out -= np.repeat(m.zeros.cpu().numpy().astype(np.float64), m.group, 1)
    return torch.from_numpy(out)


def scales_of(m):
    return m.scales.cpu().double().repeat_interleave(m.group, 1)


def columns_of(a, T, K):
    b = a.cpu().numpy().reshape(T, K // 32, 36)
    q = b[:, :, :32].copy().view(np.int8).astype(np.float64)
    d = b[:, :, 32:34].copy().view(np.float16).astype(np.float64)
    return torch.from_numpy((q * d).reshape(T, K))


def check_mm(m, a, T):
    y = torch.full((T, m.N), float("nan"), device="cuda")
    assert bqm.mm_q4(m, a, out=y) is y or True
    w, c = (steps_of(m) * scales_of(m)).cuda(), columns_of(a, T, m.K).cuda()
    want, terms = c @ w.t().contiguous(), c.abs() @ w.abs().t().contiguous()
    off = (y.double() - want).abs()
    assert bool((off <= 1e-5 * terms).all()), (float((off / terms).max()), torch.nonzero(~(off <= 1e-5 * terms))[:5])
    return y


SHAPES = [(1, 32, 32), (5, 32, 32), (16, 64, 64), (33, 128, 32), (130, 128, 128), (257, 192, 64), (100, 1024, 64),
          (65, 1120, 32), (48, 2048, 128), (31, 2080, 32), (200, 4096, 32), (513, 4096, 128), (19, 4224, 128),
          (64, 8192, 64), (7, 16416, 32), (3, 65536, 128)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 16, 17, 33, 64, 100])
@pytest.mark.parametrize("N,K,group", SHAPES)
def test_mm_q4(N, K, group, T, zeros):
    m = make_matrix(N, K, group, zeros, seed=N + K)
    check_mm(m, bqm.q8_1_quantize(randn(T, K, seed=T, scale=3.0)), T)


@pytest.mark.parametrize("T", [129, 500, 2047])
@pytest.mark.parametrize("N,K,group,zeros", [(1000, 576, 32, True), (777, 4096, 64, False), (2049, 1024, 128, True)])
def test_mm_q4_many_columns(N, K, group, zeros, T):
    check_mm(make_matrix(N, K, group, zeros, seed=T), bqm.q8_1_quantize(randn(T, K, seed=T)), T)


@pytest.mark.parametrize("T", [1, 3, 8, 20, 150])
def test_mm_q4_long_rows(T):
    check_mm(make_matrix(9, 1 << 20, 128, True, seed=T), bqm.q8_1_quantize(randn(T, 1 << 20, seed=T)), T)


@pytest.mark.parametrize("T", [1, 4, 17, 80])
def test_mm_q4_extremes(T):
    # every product at its largest, of both signs, and a column of zeros
    N, K = 40, 512
    m = make_matrix(N, K, 32, True, seed=1)
    m.codes[:20] = 0x88  # -8
    m.codes[20:] = 0x77
    m.zeros[:20], m.zeros[20:] = 7, -8
    x = torch.full((T, K), 1000.0, device="cuda")
    x[:, ::2] *= -1.0 if T > 1 else 1.0
    x[T - 1] = 0.0 if T > 1 else 1.0
    check_mm(m, bqm.q8_1_quantize(x), T)


def test_mm_q4_columns_and_rows_alone():
    # no column's or row's result depends on the others': NaN and infinity stay where they are
    m = make_matrix(70, 256, 64, False, seed=3)
    a = bqm.q8_1_quantize(randn(40, 256, seed=4))
    y = bqm.mm_q4(m, a)
    m.scales[11, 1] = float("nan")
    m.scales[12, 0] = float("inf")
    b = a.clone()
    b.view(40, 8, 36)[5, 3, 32:34] = torch.tensor([0xff, 0x7f], device="cuda", dtype=torch.uint8)  # NaN
    z = bqm.mm_q4(m, b)
    bad = ~torch.isfinite(z)
    assert bad[5].all() and bad[:, 11:13].all()
    bad[5] = False
    bad[:, 11:13] = False
    assert not bad.any()
    rest = torch.ones_like(z, dtype=torch.bool)
    rest[5] = False
    rest[:, 11:13] = False
    assert torch.equal(z[rest], y[rest])


def test_matrix_past_4_gib():
    # a table whose last rows lie past 32-bit byte offsets: the same as those rows alone
    N, K, group = 1100003, 8192, 64
    codes = torch.empty(N, K // 2, device="cuda", dtype=torch.uint8)
    scales = torch.empty(N, K // group, device="cuda", dtype=F16)
    zeros = torch.empty(N, K // group, device="cuda", dtype=torch.int8)
    part = make_matrix(257, K, group, True, seed=5)
    codes[-257:], scales[-257:], zeros[-257:] = part.codes, part.scales, part.zeros
    codes[:-257], scales[:-257], zeros[:-257] = 0, 0, 0
    big = bqm.Q4Matrix(codes, scales, zeros)
    for T in (1, 5, 17):
        a = bqm.q8_1_quantize(randn(T, K, seed=T))
        y = bqm.mm_q4(big, a)
        assert bool((y[:, :-257] == 0).all())
        w, c = (steps_of(part) * scales_of(part)).cuda(), columns_of(a, T, K).cuda()
        off = (y[:, -257:].double() - c @ w.t().contiguous()).abs()
        assert bool((off <= 1e-5 * (c.abs() @ w.abs().t().contiguous())).all())
    ids = torch.arange(257, device="cuda", dtype=torch.int32)
    assert torch.equal(bqm.q4_dequantize(big, ids + (N - 257)), bqm.q4_dequantize(part, ids))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("N,K,group,zeros", [(1, 32, 32, False), (50, 64, 64, True), (33, 480, 32, True), (129, 4096, 128, False),
                                             (20, 8320, 64, True)])
def test_q4_rows(N, K, group, zeros, dtype):
    m = make_matrix(N, K, group, zeros, seed=K)
    values = (steps_of(m) * scales_of(m)).float().cuda()  # exact: 15 bits
    for scale in (1.0, math.sqrt(K)):
        want = (values * torch.tensor(scale, dtype=F32, device="cuda")).to(dtype)
        assert torch.equal(bqm.q4_dequantize(m, scale=scale, dtype=dtype), want)
        ids = torch.randint(0, N, (77,), device="cuda", dtype=torch.int32)
        ids[3:6] = ids[0]
        assert torch.equal(bqm.q4_dequantize(m, ids, scale=scale, dtype=dtype), want[ids.long()])
    far = torch.tensor([-1, N, 2 ** 31 - 1, -2 ** 31], device="cuda", dtype=torch.int32)
    got = bqm.q4_dequantize(m, far, dtype=dtype)
    assert torch.equal(got, values.to(dtype)[[0, N - 1, N - 1, 0]])
    assert bqm.q4_dequantize(m, far[:0]).shape == (0, K)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (7, 96, 32), (30, 640, 64), (65, 1024, 128)])
def test_q4_quantize(N, K, group, zeros, dtype):
    x = randn(N, K, seed=K, dtype=dtype, scale=2.0)
    if zeros:
        x = (x.float() + 1.5).to(dtype)
    x[0, :group] = 0.0
    if N > 5:
        x[1, :group] = 4.0
        x[2, :group] *= 1e-6       # a subnormal scale
        x[3, :group] = -0.25
        if dtype != F16:
            x[4, :group] *= 1e7    # a scale past float16's range
    m = bqm.q4_quantize(x, group=group, zeros=zeros)
    assert (m.N, m.K, m.group) == (N, K, group) and (m.zeros is not None) == zeros
    g = x.cpu().float().view(N, K // group, group)
    hi, lo = g.amax(-1).clamp(min=0), g.amin(-1).clamp(max=0)
    s = (hi - lo) / 15.0 if zeros else torch.maximum(hi, -lo) / 7.0
    s16 = s.clamp(max=65504.0).half()
    assert torch.equal(m.scales.cpu(), s16)
    s = s16.float()
    some = s != 0
    div = torch.where(some, s, 1.0)
    z = torch.where(some, (-8 - torch.round(lo / div)).clamp(-8, 7), 0.0) if zeros else torch.zeros_like(s)
    if zeros:
        assert torch.equal(m.zeros.cpu(), z.to(torch.int8))
    c = torch.where(some[..., None], (torch.round(g / div[..., None]) + z[..., None]).clamp(-8, 7), 0.0)
    got = steps_of(m).view(N, K // group, group) + z[..., None].double()
    assert torch.equal(got, c.double())
    # and the values come back to within half a step where nothing was clamped
    back = bqm.q4_dequantize(m, dtype=F32).cpu().view(N, K // group, group)
    free = (c > -8) & (c < 7)
    assert bool(((back - g).abs() <= (0.5 + 8 * H32) * s[..., None])[free].all())


def test_q4_refuses():
    m = make_matrix(6, 128, 64, True, seed=1)
    a = bqm.q8_1_quantize(randn(3, 128, seed=1))
    for codes, scales, zeros, err in (
            (m.codes.cpu(), m.scales, None, TypeError), (m.codes, m.scales.float(), None, TypeError),
            (m.codes, m.scales[:5], None, ValueError), (m.codes[:, ::2], m.scales, None, ValueError),
            (m.codes, m.scales, m.zeros.short(), TypeError), (m.codes, m.scales, m.zeros[:, :1], ValueError),
            (m.codes, torch.empty(6, 0, device="cuda", dtype=F16), None, ValueError)):
        with pytest.raises(err):
            bqm.Q4Matrix(codes, scales, zeros)
    for f, err in ((lambda: bqm.mm_q4(m, a[:, :-4]), ValueError), (lambda: bqm.mm_q4(m, a.float()), TypeError),
                   (lambda: bqm.mm_q4(m, a, out=torch.empty(2, 6, device="cuda")), ValueError),
                   (lambda: bqm.mm_q4(m, a, out=torch.empty(3, 6, device="cuda", dtype=F16)), TypeError),
                   (lambda: bqm.q4_dequantize(m, torch.zeros(3, device="cuda")), TypeError),
                   (lambda: bqm.q4_dequantize(m, torch.zeros(3, 3, device="cuda", dtype=torch.int32)), ValueError),
                   (lambda: bqm.q4_dequantize(m, dtype=torch.float64), TypeError),
                   (lambda: bqm.q4_quantize(randn(4, 96, seed=1)), ValueError),
                   (lambda: bqm.q4_quantize(randn(4, 96, seed=1).double(), group=32), TypeError),
                   (lambda: bqm.mm_q4(bqm.Q4Matrix(m.codes, torch.empty(6, 8, device="cuda", dtype=F16)), a), bqm.BqmError)):
        with pytest.raises(err):
            f()
    assert bqm.mm_q4(m, a[:0]).shape == (0, 6)


# ---- sampling ----------------------------------------------------------------------------------------------------------

def plain_sample(logits, u, heat=1.0, k=0, p=1.0, least=0.0):
    """The definition, one row: (token, log of its share), fp64."""
    x = logits.double().cpu()
    x = torch.where(torch.isnan(x), -math.inf, x)
    order = torch.argsort(x, descending=True, stable=True)
    x = x[order]
    if not len(x) or x[0] == -math.inf:
        return -1, -math.inf
    if not heat > 0:
        return int(order[0]), 0.0
    w = (x == math.inf).double() if x[0] == math.inf else torch.exp((x - x[0]) / heat)
    w[x == -math.inf] = 0.0
    if k > 0:
        w[k:] = 0.0
    keep = torch.ones_like(w, dtype=torch.bool)
    if not p >= 1.0:
        c = torch.cumsum(w, 0)
        keep &= c - w < p * c[-1] if p > 0 else False
    if not least <= 0:
        keep &= w >= least
    keep[0] = True
    w = w * keep
    c = torch.cumsum(w, 0)
    u = min(max(u, 0.0), 1 - 2.0 ** -24) if u == u else 0.0
    at = int((c <= u * c[-1]).sum())
    at = min(at, int((w > 0).nonzero().max()))
    while w[at] == 0:
        at -= 1
    return int(order[at]), math.log(float(w[at]) / float(c[-1]))


def check_sample(logits, u, heat=None, k=None, p=None, least=None):
    T, V = logits.shape
    vec = lambda v, t=F32: None if v is None else torch.tensor(v, device="cuda", dtype=t)  # noqa: E731
    tokens, logprobs = bqm.sample(logits, vec(u), temperature=vec(heat), top_k=vec(k, torch.int32), top_p=vec(p), min_p=vec(least))
    as32 = lambda v, i, d: d if v is None else float(np.float32(v[i]))  # noqa: E731
    for i in range(T):
        token, lp = plain_sample(logits[i], as32(u, i, 0), as32(heat, i, 1.0), 0 if k is None else k[i], as32(p, i, 1.0),
                                 as32(least, i, 0.0))
        assert int(tokens[i]) == token, (i, int(tokens[i]), token)
        # weights below 2^-45 are left out, each other one is off by 2^-33 of itself and 2^-45 of the largest
        room = 2.0 ** -32 + V * 2.0 ** -44 + H32 * abs(lp) if math.isfinite(lp) else 0.0
        assert lp == float(logprobs[i]) or abs(float(logprobs[i]) - lp) <= room, (i, float(logprobs[i]), lp)
    return tokens


US = [0.0, 0.1, 0.37, 0.5, 0.73, 0.9, 0.999, 1 - 2.0 ** -24]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("V", [1, 2, 7, 63, 64, 65, 1000, 1023, 2049, 32001, 131071])
def test_sample_sizes(V, dtype):
    x = randn(8, V, seed=V, dtype=dtype, scale=2.5)
    check_sample(x, US)
    check_sample(x, US, heat=[0.5, 0.7, 1.0, 1.0, 1.3, 2.0, 0.1, 5.0])
    check_sample(x, US, k=[1, 2, 5, 50, 1000, V, V + 9, 0])
    check_sample(x, US, p=[0.0, 0.1, 0.5, 0.9, 0.95, 0.999, 1.0, 2.0])
    check_sample(x, US, least=[0.0, 1e-6, 0.01, 0.05, 0.1, 0.5, 1.0, 2.0])
    check_sample(x, US, heat=[0.0, 0.7, 1.0, 1.0, 1.3, 2.0, -1.0, 1.0], k=[0, 40, 0, 100, 2000, 0, 5, 3000],
                 p=[1.0, 0.9, 0.95, 1.0, 0.8, 0.99, 0.9, 0.7], least=[0.1, 0.0, 0.02, 0.1, 0.0, 1e-4, 0.0, 1e-3])


@pytest.mark.parametrize("V", [5000, 131071])
def test_sample_many_equal(V):
    # all logits equal; two values; a ladder of neighbouring floats: bins that cannot be sorted as a whole
    x = torch.zeros(8, V, device="cuda")
    more = dict(k=[0, 1, 3000, 0, V // 2, 0, 0, 4000], p=[1.0, 1.0, 1.0, 0.5, 0.5, 0.9, 1.0, 0.25])
    check_sample(x, US)
    check_sample(x, US, **more)
    x[:, 1::3] = -0.5
    x[:, 2::3] = -0.0
    check_sample(x, US, **more)
    ladder = (torch.randperm(V, generator=torch.Generator().manual_seed(1)).cuda().float() * 2.0 ** -23 + 1.0).expand(8, V).contiguous()
    check_sample(ladder, US, **more)
    check_sample(ladder.to(BF16), US, **more)
    ladder[:, ::2] = 3.0
    check_sample(ladder, US, **more)


def test_sample_masks():
    inf, nan = math.inf, math.nan
    x = randn(8, 3000, seed=1)
    x[:, ::2] = -inf
    x[1] = -inf
    x[2] = -inf
    x[2, 1234] = -60000.0
    x[3, 5::10] = nan
    x[4] = nan
    x[5, 100:103] = inf
    x[6] = torch.finfo(F32).min
    x[7] = torch.finfo(F32).min
    x[7, 17] = torch.finfo(F32).max
    t = check_sample(x, US)
    assert t[1] == -1 and t[4] == -1 and t[2] == 1234 and 100 <= t[5] < 103 and t[7] == 17
    check_sample(x, US, k=[50] * 8, p=[0.9] * 8, least=[0.01] * 8)
    check_sample(x, US, heat=[0.0] * 8)
    check_sample(x, US, heat=[inf] * 8)
    check_sample(x, US, heat=[1e-30] * 8)


def test_sample_odd_settings():
    x = randn(8, 900, seed=2)
    check_sample(x, [-1.0, math.nan, 1.0, 2.0, math.inf, -math.inf, 0.3, 0.4])
    check_sample(x, US, k=[-5] * 8)
    # a setting that is no number, or that leaves nothing, takes the first token
    best = x.argmax(-1).to(torch.int32)
    u = torch.tensor(US, device="cuda")
    for name, value in (("temperature", math.nan), ("temperature", -1.0), ("top_p", math.nan), ("top_p", -1.0), ("top_p", 0.0),
                        ("min_p", math.nan), ("min_p", 1.5), ("min_p", 1.0)):
        tokens, logprobs = bqm.sample(x, u, **{name: torch.full((8,), value, device="cuda")})
        assert torch.equal(tokens, best) and bool((logprobs == 0).all()), (name, value)


def test_sample_shares():
    # over evenly spaced u, every token is drawn as often as its share says, to within one draw
    n = 1 << 16
    x = randn(1, 50, seed=3, scale=1.5)
    u = (torch.arange(n, device="cuda") + 0.5) / n
    got = []
    for at in range(0, n, 32768):
        got.append(bqm.sample(x.expand(32768, 50).contiguous(), u[at:at + 32768].contiguous())[0])
    count = torch.bincount(torch.cat(got).long(), minlength=50).double() / n
    assert float((count - torch.softmax(x[0].double(), 0)).abs().max()) <= 1.0 / n + 1e-6


def test_sample_strides_and_outputs():
    wide = randn(6, 5003, seed=4)
    x = wide[:, 1:4002]
    u = torch.rand(6, device="cuda")
    tokens, lp = bqm.sample(x.contiguous(), u)
    got = bqm.sample(x, u, out=torch.full((6,), -9, device="cuda", dtype=torch.int32), logprobs=torch.full((6,), 9.0, device="cuda"))
    assert torch.equal(got[0], tokens) and torch.equal(got[1], lp)
    same = wide[:1].expand(4, 5003)
    with pytest.raises(bqm.BqmError):
        bqm.sample(same, u[:4])  # rows over one another
    t, lp = bqm.sample(wide[:0], u[:0])
    assert t.shape == (0,) and lp.shape == (0,)


def test_sample_refuses():
    x, u = randn(4, 100, seed=5), torch.rand(4, device="cuda")
    for f, err in ((lambda: bqm.sample(x.cpu(), u), TypeError), (lambda: bqm.sample(x.double(), u), TypeError),
                   (lambda: bqm.sample(x, u[:3]), ValueError), (lambda: bqm.sample(x, u.double()), TypeError),
                   (lambda: bqm.sample(x[:, ::2], u), ValueError), (lambda: bqm.sample(x[0], u), ValueError),
                   (lambda: bqm.sample(x, u, top_k=u), TypeError), (lambda: bqm.sample(x, u, top_p=u[:2]), ValueError),
                   (lambda: bqm.sample(x, u, temperature=u.cpu()), TypeError),
                   (lambda: bqm.sample(x, u, out=torch.empty(4, device="cuda", dtype=torch.int64)), TypeError),
                   (lambda: bqm.sample(torch.empty(1, 1 << 20, device="cuda"), u[:1]), bqm.BqmError)):
        with pytest.raises(err):
            f()
