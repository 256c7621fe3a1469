"""Workspaces of the token side: one made for a server's largest call serves its smaller ones."""
import ctypes

import pytest
import torch

import bit_quantized_mat_amd as bqm
from bit_quantized_mat_amd.tokens import _Q4Struct

F32, F16 = torch.float32, torch.float16


@pytest.mark.parametrize("N,K,group", [(4096, 4096, 128), (14336, 4096, 128), (5, 4096, 64), (100003, 4096, 32),
                                       (32, 65536, 128), (21760, 12288, 64), (300, 9120, 32), (4096, 1 << 20, 32),
                                       (2000, 1 << 18, 32), (65537, 544, 32)])
def test_mm_q4_workspace_never_falls(N, K, group):
    m = _Q4Struct(codes=None, scales=None, zeros=None, N=N, K=K, group=group)
    last = 0
    for T in sorted({*range(1, 2300), *range(2301, 65536, 97), 8191, 8192, 8193, 65535, 65536}):
        need = bqm.library().mm_q4_workspace_bytes(ctypes.byref(m), T)
        assert need >= last, (T, need, last)
        last = need


@pytest.mark.parametrize("V", [1, 2000, 40000, 40699, 40700, 100003, 129599, 129600, 131071, (1 << 20) - 1])
def test_sample_workspace_never_falls(V):
    last = 0
    for T in [0, *range(1, 300), *range(300, 65535, 991), 65535]:
        need = bqm.sample_workspace_bytes(T, V)
        assert need >= last, (T, need, last)
        last = need


@pytest.mark.gpu
@pytest.mark.parametrize("V", [41000, 100003])
def test_sample_in_the_workspace_of_a_larger_call(V):
    g = torch.Generator(device="cuda").manual_seed(V)
    x, u = torch.randn(256, V, generator=g, device="cuda"), torch.rand(256, generator=g, device="cuda")
    need = bqm.sample_workspace_bytes(256, V)
    room = torch.full((need + 4096,), 0xff, device="cuda", dtype=torch.uint8)
    for T in (256, 1, 2, 64, 85, 86, 128, 0):
        tokens, logprobs = bqm.sample(x[:T], u[:T], workspace=room[:need])
        assert bool((room[need:] == 0xff).all())
        want = bqm.sample(x[:T], u[:T])
        assert torch.equal(tokens, want[0]) and torch.equal(logprobs, want[1]), T


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,group", [(4096, 4096, 128), (300, 9120, 32), (40, 65536, 64)])
def test_mm_q4_in_the_workspace_of_a_larger_call(N, K, group):
    g = torch.Generator(device="cuda").manual_seed(K)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand(N, K // group, generator=g, device="cuda") - 0.3) * 0.1).half()
    m = bqm.Q4Matrix(codes, scales)
    need = bqm.mm_q4_workspace_bytes(m, 2048)
    room = torch.full((need + 4096,), 0xff, device="cuda", dtype=torch.uint8)
    a = bqm.q8_1_quantize(torch.randn(2048, K, generator=g, device="cuda"))
    for T in (2048, 1, 20, 33, 64, 128, 129, 512, 1024):
        y = bqm.mm_q4(m, a[:T], workspace=room[:need])
        assert bool((room[need:] == 0xff).all())
        assert torch.equal(y, bqm.mm_q4(m, a[:T])), T
