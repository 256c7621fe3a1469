"""NaN and infinities on the token side: where they go and where they do not."""
import pytest
import torch

import bit_quantized_mat_amd as bqm

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
INF, NAN = float("inf"), float("nan")


def test_norm_to_blocks_takes_them_as_the_quantizer_does():
    # of floats a broken row is NaN; its blocks are what q8_1_quantize makes of that, which takes a NaN as 0:
    # zeros where all of a block is NaN. No other row is touched.
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(8, 1056, generator=g, device="cuda").to(BF16)
    clean, _ = bqm.rms_norm_q8_1(x)
    x[1, 7], x[3, 1000], x[4, 5] = NAN, INF, -INF
    gain = torch.ones(1056, device="cuda")
    y, _ = bqm.rms_norm(x, gain, out_dtype=torch.float32)
    a, _ = bqm.rms_norm_q8_1(x, gain)
    assert torch.equal(a, bqm.q8_1_quantize(y))
    assert bool(torch.isnan(y[1]).all()) and bool((a[1] == 0).all())
    assert bool(torch.isnan(y[3, 1000])) and bool(torch.isnan(y[4, 5])) and not bool(a[3:5].any())
    rest = [0, 2, 5, 6, 7]
    assert torch.equal(a[rest], clean[rest])
    # some values of a block: the others are kept
    gain[40], gain[99] = NAN, -NAN
    y, _ = bqm.rms_norm(x, gain, out_dtype=torch.float32)
    a, _ = bqm.rms_norm_q8_1(x, gain)
    assert torch.equal(a, bqm.q8_1_quantize(y)) and bool(torch.isnan(y[:, 40]).all())
    blocks = a.view(8, 33, 36)
    assert not bool(blocks[:, 1, 8].any()) and not bool(blocks[:, 3, 3].any()) and bool(blocks[rest, 1, :32].any(-1).all())


@pytest.mark.parametrize("shape", [(3, 1000), (40, 80021)])
def test_rows_of_nan_are_not_drawn_from(shape):
    # what a broken row's products give: a row of NaN has no token
    x = torch.randn(*shape, device="cuda")
    u = torch.rand(shape[0], device="cuda")
    want = bqm.sample(x, u)
    x[1] = NAN
    tokens, logprobs = bqm.sample(x, u)
    assert int(tokens[1]) == -1 and float(logprobs[1]) == -INF
    keep = [i for i in range(shape[0]) if i != 1]
    assert torch.equal(tokens[keep], want[0][keep]) and torch.equal(logprobs[keep], want[1][keep])
