"""Random numbers outside [0, 1), which are clamped, where the sum of a row's weights is near 2^64."""
import pytest
import torch

import bit_quantized_mat_amd as bqm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [1000, 100003, (1 << 20) - 1])
@pytest.mark.parametrize("rows", [8, 136])
def test_numbers_outside_their_range(rows, V):
    # all logits equal, so the tokens are in the order of their ids: the last one from 1 on, the first up to 0
    x = torch.zeros(1, V, device="cuda").expand(rows, V).contiguous()
    u = [1.0, 1.0000001, 1.9, 2.0, 1e30, float("inf"), -1.0, float("nan")]
    tokens, logprobs = bqm.sample(x, torch.tensor(u * (rows // 8), device="cuda"))
    assert tokens.tolist() == ([V - 1] * 6 + [0, 0]) * (rows // 8)
    assert float((logprobs + torch.log(torch.tensor(float(V)))).abs().max()) <= 2.0 ** -23 * 14
