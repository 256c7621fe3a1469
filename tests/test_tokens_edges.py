"""The token side where its work is dealt out otherwise: sampling by one workgroup a row or by
several, products in several turns over the columns and in parts over the runs."""
import ctypes

import pytest
import torch

import bit_quantized_mat_amd as bqm
from bit_quantized_mat_amd.tokens import _Q4Struct

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def need(N, K, T):
    m = _Q4Struct(codes=None, scales=None, zeros=None, N=N, K=K, group=32)
    return bqm.library().mm_q4_workspace_bytes(ctypes.byref(m), T)


@pytest.mark.parametrize("N,K", [(21760, 1536), (21760, 4096), (300, 2048), (128, 8192), (5000, 544), (100003, 4096)])
def test_workspace_of_several_turns(N, K):
    # 8192 columns a turn: what is left for the last one has to find its own workspace
    for rest in (33, 64, 65, 128, 200, 1000, 8191, 8192):
        for turns in (1, 2, 7):
            T = 8192 * turns + rest
            if T <= 65536:
                assert need(N, K, T) >= max(need(N, K, rest), need(N, K, 8192)), (rest, turns)


def randn(*shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def matrix(N, K, group, zeros, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand(N, K // group, generator=g, device="cuda") - 0.3) * 0.1).half()
    z = torch.randint(-8, 8, (N, K // group), generator=g, device="cuda", dtype=torch.int8) if zeros else None
    return bqm.Q4Matrix(codes, scales, z)


@pytest.mark.gpu
@pytest.mark.parametrize("rest", [1, 2, 20, 33, 64, 130])
@pytest.mark.parametrize("N,K,group,zeros", [(300, 2048, 64, True), (129, 544, 32, False)])
def test_mm_q4_in_several_turns(N, K, group, zeros, rest):
    # each turn's columns as a call of theirs gives them; a last turn of up to 32 columns takes
    # other kernels than such a call: both within 1e-5 of the terms' sum, the header's bound
    T = 8192 + rest
    m = matrix(N, K, group, zeros, seed=rest)
    a = bqm.q8_1_quantize(randn(T, K, seed=N))
    # a workspace of the size asked for, inside a larger one that has to stay as it is
    bytes_ = bqm.mm_q4_workspace_bytes(m, T)
    room = torch.full((bytes_ + 4096,), 0xa5, device="cuda", dtype=torch.uint8)
    y = bqm.mm_q4(m, a, workspace=room[:bytes_])
    assert bool((room[bytes_:] == 0xa5).all())
    assert torch.equal(y[:8192], bqm.mm_q4(m, a[:8192]))
    one = bqm.mm_q4(m, a[8192:])
    if rest > 32:
        assert torch.equal(y[8192:], one)
    else:
        w = bqm.q4_dequantize(m, dtype=F32).double()
        b = a[8192:].view(rest, K // 32, 36).contiguous()
        q = b[:, :, :32].contiguous().view(torch.int8).double()
        d = b[:, :, 32:34].contiguous().view(F16).double()
        c = (q * d).view(rest, K)
        # (dequantized values are rounded to fp32: 2^-24 of each)
        room = (1e-5 + 2.0 ** -24) * (c.abs() @ w.abs().t().contiguous())
        want = c @ w.t().contiguous()
        assert bool(((y[8192:].double() - want).abs() <= room).all())
        assert bool(((one.double() - want).abs() <= room).all())


SETTINGS = [dict(), dict(heat=[0.5, 0.7, 1.0, 1e-4, 1.3, 2.0, 0.1, 5.0]),
            dict(k=[1, 2, 5, 50, 1000, 4000, 0, 200000]), dict(p=[0.0, 0.1, 0.5, 0.9, 0.95, 0.999, 1.0, 2.0]),
            dict(least=[0.0, 1e-6, 0.01, 0.05, 0.1, 0.5, 1.0, 2.0]),
            dict(heat=[0.0, 0.7, 1.0, 1.0, 1.3, 2.0, -1.0, 1.0], k=[0, 40, 0, 100, 2000, 0, 5, 3000],
                 p=[1.0, 0.9, 0.95, 1.0, 0.8, 0.99, 0.9, 0.7], least=[0.1, 0.0, 0.02, 0.1, 0.0, 1e-4, 0.0, 1e-3])]


def draw(x, times, heat=None, k=None, p=None, least=None):
    vec = lambda v, t=F32: None if v is None else torch.tensor(v * times, device="cuda", dtype=t)  # noqa: E731
    u = [0.0, 0.1, 0.37, 0.5, 0.73, 0.9, 0.999, 1 - 2.0 ** -24]
    return bqm.sample(x.repeat(times, 1), vec(u), temperature=vec(heat), top_k=vec(k, torch.int32), top_p=vec(p),
                      min_p=vec(least))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("V", [4097, 32001, 45600, 131071, 262143])
@pytest.mark.parametrize("kind", ["normal", "equal", "ladder", "masked"])
def test_sample_does_not_depend_on_the_number_of_rows(kind, V, dtype):
    # from 45600 logits on 8 rows have several workgroups each, 64 fewer, 129 and more one: the same bits
    if kind == "normal":
        x = randn(8, V, seed=V, dtype=dtype, scale=2.5)
    elif kind == "equal":
        x = torch.zeros(8, V, device="cuda", dtype=dtype)
        x[:, 1::3] = -0.5
    elif kind == "ladder":
        x = (torch.arange(V, device="cuda").float().flip(0) * 2.0 ** -23 + 1.0).expand(8, V).to(dtype)
    else:
        x = randn(8, V, seed=V + 1, dtype=dtype)
        x[:, V // 3:] = float("-inf")
        x[1] = float("-inf")
        x[2, ::2] = float("nan")
        x[3, 7::1000] = float("inf")
        x[4] = torch.finfo(dtype).min
    for settings in SETTINGS:
        tokens, logprobs = draw(x, 1, **settings)
        assert bool((tokens < V).all()) and bool((tokens >= (0 if kind != "masked" else -1)).all())
        for times in (8, 16, 17):
            got = draw(x, times, **settings)
            assert torch.equal(got[0], tokens.repeat(times)), (times, settings)
            assert torch.equal(got[1], logprobs.repeat(times)), (times, settings)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 256, 288, 512])
@pytest.mark.parametrize("T", [1, 7, 64, 1001])
def test_norm_of_short_rows(T, K):
    # several rows a wave: heads' norms. fp32 throughout: r, s * r and its product with gain are
    # rounded, 2^-24 each
    x, add, gain = randn(T, K, seed=T, dtype=BF16, scale=2.0), randn(T, K, seed=K), randn(K, seed=3)
    x[T // 2] = 0.0
    add[T // 2] = 0.0
    s = (x.float() + add).to(BF16)
    y, got = bqm.rms_norm(x, gain, add=add, out_dtype=F32)
    assert torch.equal(got, s)
    d = s.double()
    want = d / (d.square().mean(-1, keepdim=True) + 1e-6).sqrt() * gain.double()
    room = ((1 + 2.0 ** -24) ** 3 - 1 + 2.0 ** -45) * want.abs() + 2.0 ** -148
    assert bool(((y.double() - want).abs() <= room).all())
    a, _ = bqm.rms_norm_q8_1(x, gain, add=add)
    assert torch.equal(a, bqm.q8_1_quantize(y))
    # each row as it is alone
    for t in {0, T // 2, T - 1}:
        one, _ = bqm.rms_norm(x[t:t + 1], gain, add=add[t:t + 1], out_dtype=F32)
        assert torch.equal(one, y[t:t + 1])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 20])
@pytest.mark.parametrize("K,group,zeros", [(32, 32, True), (544, 32, False), (1152, 128, True), (2112, 64, False)])
@pytest.mark.parametrize("N", [16, 4111, 8200, 12300, 28688, 30001, 45007, 66001])
def test_mm_q4_rows_shared_by_waves(N, K, group, zeros, T):
    # one tile a workgroup to dozens, tiles of which waves have a part: the header's bound
    m = matrix(N, K, group, zeros, seed=N)
    a = bqm.q8_1_quantize(randn(T, K, seed=K, scale=2.0))
    y = bqm.mm_q4(m, a, out=torch.full((T, N), float("nan"), device="cuda"))
    w = bqm.q4_dequantize(m, dtype=F32).double()
    b = a.view(T, K // 32, 36)
    c = (b[:, :, :32].contiguous().view(torch.int8).double() * b[:, :, 32:34].contiguous().view(F16).double()).view(T, K)
    # (dequantized values are rounded to fp32: 2^-24 of each)
    room = (1e-5 + 2.0 ** -24) * (c.abs() @ w.abs().t().contiguous())
    assert bool(((y.double() - c @ w.t().contiguous()).abs() <= room).all())


@pytest.mark.gpu
def test_more_workgroups_than_a_row_of_the_grid():
    # above 2^20 workgroups the grid has a second dimension: rows behind that are right, and the
    # last place's neighbour stays as it was
    T, K = (1 << 21) + 3, 1024  # two rows a workgroup
    x = torch.empty(T, K, device="cuda", dtype=BF16).fill_(1.0)
    few = randn(5, K, seed=1, dtype=BF16)
    x[-5:] = few
    y, _ = bqm.rms_norm(x)
    assert torch.equal(y[-5:], bqm.rms_norm(few)[0]) and torch.equal(y[:1], bqm.rms_norm(x[:1])[0])
    assert torch.equal(y[:-5], y[:1].expand(T - 5, K))
    del y
    m = bqm.q4_quantize(x, group=32, zeros=True)  # 256 threads of eight values: 2^20 and more workgroups
    want = bqm.q4_quantize(few, group=32, zeros=True)
    assert torch.equal(m.codes[-5:], want.codes) and torch.equal(m.scales[-5:], want.scales)
    assert torch.equal(m.zeros[-5:], want.zeros) and torch.equal(m.codes[:-5], m.codes[:1].expand(T - 5, K // 2))
    del x
    out = torch.full(((1 << 22) + 9, K), 7.0, device="cuda", dtype=F16)  # four rows a workgroup
    ids = torch.full(((1 << 22) + 8,), T - 1, device="cuda", dtype=torch.int32)
    ids[-1] = T - 5
    bqm.q4_dequantize(m, ids, out=out[:-1])
    rows = bqm.q4_dequantize(want, dtype=F16)
    assert torch.equal(out[-2], rows[0]) and bool((out[-1] == 7.0).all())
    assert torch.equal(out[:-2], rows[4:].expand((1 << 22) + 7, K))
    del out
    # products of one and two columns: 1024 rows of 32 values a workgroup
    N = (1 << 30) + 2048
    codes = torch.zeros(N, 16, device="cuda", dtype=torch.uint8)
    scales = torch.ones(N, 1, device="cuda", dtype=F16)
    codes[-1] = 0x11
    a = bqm.q8_1_quantize(torch.full((2, 32), 127.0, device="cuda"))
    for t in (1, 2):
        y = bqm.mm_q4(bqm.Q4Matrix(codes, scales), a[:t])
        assert bool((y[:, :-1] == 0).all()) and bool((y[:, -1] == 32 * 127.0).all())
        del y
