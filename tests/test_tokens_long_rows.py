"""Products of 4-bit matrices with long rows: the header's bound, 1e-5 of the sum of the terms'
absolute values, where every rounding goes the same way. Inputs are made so that sums are known
exactly, and so that one fp32 sum over all of a row's groups misses the bound."""
import ctypes

import numpy as np
import pytest
import torch

import bit_quantized_mat_amd as bqm
from bit_quantized_mat_amd.tokens import _Q4Struct

F32, F16 = torch.float32, torch.float16


def blocks(q_sum, d):
    """Q8_1 blocks of one column: run j holds whole numbers of sum q_sum[j] and the scale d[j]."""
    nb = len(q_sum)
    b = np.zeros((nb, 36), np.uint8)
    q = b[:, :32].view(np.int8)
    for j in {*q_sum}:
        rest, at = j, q_sum == j
        for i in range(32):
            q[at, i] = (rest + 31 - i) // (32 - i)
            rest -= (rest + 31 - i) // (32 - i)
    b[:, 32:34] = np.asarray(d, np.float16).reshape(nb, 1).view(np.uint8)
    b[:, 34:36] = (np.asarray(d, np.float64) * q_sum).astype(np.float16).reshape(nb, 1).view(np.uint8)
    return b.reshape(-1)


def ones(N, K, group, zeros, scale=1.0):
    """A matrix whose every value is scale."""
    z = torch.ones(N, K // group, device="cuda", dtype=torch.int8) if zeros else None
    codes = torch.full((N, K // 2), 0x22 if zeros else 0x11, device="cuda", dtype=torch.uint8)
    return bqm.Q4Matrix(codes, torch.full((N, K // group), scale, device="cuda", dtype=F16), z)


def check(m, column, T, want):
    y = bqm.mm_q4(m, torch.from_numpy(column).cuda().expand(T, -1).contiguous())
    lo, hi = float(y.min()), float(y.max())
    assert abs(lo - want) <= 1e-5 * want and abs(hi - want) <= 1e-5 * want, (lo / want - 1, hi / want - 1)


def one_and_little(K, group, first):
    """The column and its sum: `first` runs of 32, then a run a group just above half of 32's last
    place, which a sum of 32 rounds up to a whole one: 2^-24 of 32 each."""
    nb = K // 32
    q, d = np.zeros(nb, np.int64), np.full(nb, 2.0 ** -24)
    q[::group // 32] = 33
    q[:first], d[:first] = 32, 1.0
    return blocks(q, d), float((q * d).sum())


# kernels: of one and two columns (64 lanes a row, each its own sum), of the few that fit in LDS, of tiles of
# 32, 64 and 128 columns; rows so many that no kernel cuts them by itself
@pytest.mark.gpu
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N,K,group,T,first", [
    (70, 1 << 20, 32, 1, 64), (70, 1 << 20, 32, 2, 64), (33, 1 << 19, 32, 1, 64), (9, 1 << 20, 128, 2, 64),
    (65536, 9088, 32, 3, 1), (28671, 9088, 32, 16, 1), (65536, 6016, 32, 9, 1), (30000, 4480, 32, 32, 1), (30000, 4544, 32, 32, 1),
    (65536, 9088, 64, 5, 1), (28671, 9088, 128, 16, 1),
    (21888, 16384, 32, 40, 1), (21888, 16384, 32, 20, 1), (21888, 32768, 64, 64, 1), (14336, 32768, 32, 256, 1),
    (2816, 65536, 32, 1024, 1), (2816, 1 << 18, 128, 1024, 1), (2816, 1 << 20, 32, 1024, 1), (21888, 65568, 32, 33, 1)])
def test_roundings_of_one_side(N, K, group, T, first, zeros):
    column, want = one_and_little(K, group, first)
    check(ones(N, K, group, zeros), column, T, want)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,group,T", [(14336, 32768, 32, 256), (2816, 65536, 32, 1024), (2816, 1 << 20, 32, 1024),
                                         (2816, 1 << 20, 128, 1024), (40, 1 << 20, 32, 150), (40, 1 << 20, 32, 1)])
def test_equal_terms(N, K, group, T):
    scale, d = np.float16(0.1), np.float16(0.3)
    nb = K // 32
    column = blocks(np.full(nb, 32 * 77), np.full(nb, d))
    check(ones(N, K, group, False, float(scale)), column, T, float(scale) * float(d) * 32 * 77 * nb)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,group,zeros,T", [(2811, 70016, 32, True, 1000), (2811, 300288, 32, True, 1000), (2811, 20512, 32, False, 1000),
                                               (21999, 12320, 32, True, 40), (22001, 24640, 64, True, 70),
                                               (22001, 35200, 128, False, 35), (1400, 140032, 64, True, 2047)])
def test_ragged_long_rows(N, K, group, zeros, T):
    g = torch.Generator(device="cuda").manual_seed(K)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand(N, K // group, generator=g, device="cuda") - 0.3) * 0.1).half()
    z = torch.randint(-8, 8, (N, K // group), generator=g, device="cuda", dtype=torch.int8) if zeros else None
    m = bqm.Q4Matrix(codes, scales, z)
    a = bqm.q8_1_quantize(torch.randn(T, K, generator=g, device="cuda"))
    out = torch.full((T + 2, N), 7.0, device="cuda")
    y = bqm.mm_q4(m, a, out=out[1:-1])
    assert bool((out[0] == 7).all()) and bool((out[-1] == 7).all())
    b = a.view(T, K // 32, 36)
    c = (b[:, :, :32].contiguous().view(torch.int8).double() * b[:, :, 32:34].contiguous().view(F16).double()).view(T, K)
    rows = torch.cat((torch.arange(0, N, 37), torch.arange(N - 9, N))).to(torch.int32).cuda()
    w = bqm.q4_dequantize(m, rows, dtype=F32).double()
    # (dequantized values are rounded to fp32: 2^-24 of each)
    room = (1e-5 + 2.0 ** -24) * (c.abs() @ w.abs().t().contiguous())
    assert bool(((y[:, rows.long()].double() - c @ w.t().contiguous()).abs() <= room).all())
    assert torch.equal(bqm.mm_q4(m, a), y)


def test_workspace_of_long_rows():
    # rows longer than any way of adding up one part's sums allows have further parts' sums, whatever the
    # number of rows and columns; others none where those give work enough
    N, T = 100003, 1000

    def sums(K, group):
        m = _Q4Struct(codes=None, scales=None, zeros=None, N=N, K=K, group=group)
        laid = 32 * -(-K // 128) * 4 * (2048 + 128)  # columns as operands and their scales
        return bqm.library().mm_q4_workspace_bytes(ctypes.byref(m), T) - laid

    for group in (32, 64, 128):
        assert sums(2048 * group, group) == 0
        assert sums(1 << 20, group) >= 2 * T * N * 4 and sums(1 << 20, group) % (T * N * 4) == 0
