"""Launches of few rows (single tokens, short drafts): how many bits their weights keep."""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_attention import Setup, UNIT, _attention64, _f64  # noqa: E402


@pytest.fixture(scope="module")
def bqm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_mat_amd as m
    m.library()
    return m


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lens,q_lens,H,Hq,D,window", [
    ([5], [1], 1, 4, 64, 0), ([37], [1], 8, 32, 128, 0), ([12, 0, 31], [8, 1, 3], 2, 8, 72, 0),
    ([3000], [1], 1, 4, 128, 0), ([70], [4], 1, 2, 256, 16), ([6000, 40], [2, 2], 2, 2, 64, 0),
])
def test_weights_keep_twice_the_types_bits(bqm, lens, q_lens, H, Hq, D, window, dt):
    print("few rows", lens, q_lens, H, Hq, D, window, dt, file=sys.stderr, flush=True)
    s = Setup(lens, q_lens, H, D, 16, dt, seed=50, n_q=Hq)
    scale = D ** -0.5
    y = _f64(bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), s.batch(bqm, max_q=max(q_lens)), window=window,
                                 out_dtype=torch.float32))
    want, mean, seen, spread = _attention64(s, scale, True, window)
    # a weight's rounding leaves u of it, that rest's rounding u of the rest (or, in
    # float16, 2^-32 of the row's largest weight); the scores, the exponential and the
    # sums as everywhere in 32 bits
    vmax = max(float(v.abs().max()) for v in s.vs if len(v))
    rel = UNIT[dt] ** 2 + 2.0 * ((D + 16) * 2.0 ** -23 * spread + 2.0 ** -20) + seen * 2.0 ** -23
    bound = rel[..., None] * mean * 1.02 + 2.0 ** -24 * np.abs(want)
    bound += (seen * vmax * (2.0 ** -32 if dt == "f16" else 0.0))[..., None]
    err = np.abs(y - want)
    assert np.all(err <= bound), float((err - bound).max())
    assert np.all(y[seen == 0] == 0.0)
