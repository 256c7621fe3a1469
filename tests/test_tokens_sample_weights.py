"""Sampling's weights, as exactly as the header states them: within 2^-32 of themselves."""
import numpy as np
import pytest
import torch

import bit_quantized_mat_amd as bqm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heat", [1.0, 0.7, 3.3])
def test_weights_beside_a_border(heat):
    # rows [0, v] whose second weight is 2^-31.9 to 2^-31 of itself above or below min_p, a fp32 number: it
    # has to stay or go as it does in 64 bits (exp in fp64 is off by 2^-52)
    heat = np.float32(heat)
    rng = np.random.default_rng(5)
    v = -rng.random(6_000_000, np.float32) * np.float32(2.5) * heat
    w = np.exp(v.astype(np.float64) / float(heat))
    floor = w.astype(np.float32)
    off = w / floor - 1.0
    near = np.flatnonzero((np.abs(off) > 2.0 ** -31.9) & (np.abs(off) < 2.0 ** -31))[:65535]
    assert len(near) > 4000 and (off[near] > 0).any() and (off[near] < 0).any()
    n = len(near)
    x = torch.zeros(n, 2, device="cuda")
    x[:, 1] = torch.from_numpy(v[near]).cuda()
    full = lambda f: torch.full((n,), float(f), device="cuda")  # noqa: E731
    # u of the whole lies past the first weight, 1, if the second is there
    tokens, logprobs = bqm.sample(x, full(0.95), temperature=full(heat), min_p=torch.from_numpy(floor[near]).cuda())
    stays = torch.from_numpy(off[near] > 0).cuda()
    assert torch.equal(tokens == 1, stays)
    w = torch.from_numpy(w[near]).cuda()
    want = torch.where(stays, torch.log(w) - torch.log1p(w), 0.0)
    # a log-share is off by the weight's 2^-32 and its rounding to fp32
    assert bool(((logprobs.double() - want).abs() <= 2.0 ** -31 + 2.0 ** -24 * want.abs()).all())
