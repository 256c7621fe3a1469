"""Products of 4-bit matrices: NaN and infinite scales in each kernel, the output given."""
import pytest
import torch

import bit_quantized_mat_amd as bqm

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def matrix(n, k, group, zeros, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand(n, k // group, generator=g, device="cuda") + 0.1) * 0.1).half()
    z = torch.randint(-8, 8, (n, k // group), generator=g, device="cuda", dtype=torch.int8) if zeros else None
    return bqm.Q4Matrix(codes, scales, z)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N,K,group", [(70, 256, 64), (70, 288, 32), (5000, 512, 128), (70, 4096, 32), (66, 9216, 128)])
@pytest.mark.parametrize("T", [1, 2, 3, 9, 16, 17, 32, 33, 65, 130])
def test_products_keep_them_in_their_rows_and_columns(T, N, K, group, zeros):
    # one and two columns, few in LDS, tiles in one part and in several
    m = matrix(N, K, group, zeros, seed=K)
    a = bqm.q8_1_quantize(torch.randn(T, K, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda"))
    y = bqm.mm_q4(m, a)
    rows = [0, 11, 12, N - 1]
    m.scales[0, 0], m.scales[11, -1], m.scales[12, 1], m.scales[N - 1, 0] = NAN, NAN, INF, -INF
    b = a.clone()
    if T > 1:
        b.view(T, K // 32, 36)[T - 1, 3, 32:34] = torch.tensor([0xff, 0x7f], device="cuda", dtype=torch.uint8)  # NaN
    z = bqm.mm_q4(m, b)
    bad = torch.zeros(T, N, device="cuda", dtype=torch.bool)
    bad[:, rows] = True
    if T > 1:
        bad[T - 1] = True
    # (an infinite scale's group sums to 0 here or there: NaN, no finite value either)
    assert not bool(torch.isfinite(z[bad]).any())
    assert torch.equal(z[~bad], y[~bad])


@pytest.mark.parametrize("T", [1, 2, 20, 40])
def test_the_output_given_is_the_one_returned(T):
    m = matrix(40, 128, 64, False, seed=1)
    a = bqm.q8_1_quantize(torch.randn(T, 128, device="cuda"))
    out = torch.full((T, 40), NAN, device="cuda")
    y = bqm.mm_q4(m, a, out=out)
    assert y.data_ptr() == out.data_ptr() and y.shape == out.shape and torch.equal(out, bqm.mm_q4(m, a))
