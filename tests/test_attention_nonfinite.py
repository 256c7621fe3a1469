"""Attention where values, keys or queries are infinite, NaN or as large as their
type holds, and where weights are far below the largest: each row gets what it
sees, and nothing of what it does not."""
import math
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_attention import DT, Setup, UNIT, _close_attention, _f64, _ints  # noqa: E402

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def bqm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_mat_amd as m
    m.library()
    return m


def _diagonal_infinities(s, first):
    """Value i of token first + i becomes infinite, for every value i of a head: one
    token at each place of a wave's 64."""
    for i in range(s.D):
        j = first + i
        s.v[int(s.table[0, j // s.ps]), j % s.ps, :, i] = INF


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("n,nan_at", [(64, 40), (128, 100), (130, 90)])
def test_infinities_beside_rows_of_a_nan_key(bqm, n, nan_at, dt):
    # rows from nan_at on see a NaN key; the rows before them in the same tile do
    # not, and get every infinity they see
    print("nan key", n, nan_at, dt, file=sys.stderr, flush=True)
    s = Setup([n], [n], 1, 64, 16, dt, seed=40)
    cache = bqm.KvCache(s.k, s.v)
    clean = bqm.paged_attention(s.q, cache, s.batch(bqm))
    _diagonal_infinities(s, 0)
    s.k[int(s.table[0, nan_at // 16]), nan_at % 16] = NAN
    y = bqm.paged_attention(s.q, cache, s.batch(bqm))[:, 0]
    row, col = torch.arange(n, device="cuda")[:, None], torch.arange(64, device="cuda")[None]
    assert torch.isnan(y[nan_at:]).all()
    sees = (col <= row)[:nan_at]
    assert torch.isposinf(y[:nan_at][sees]).all()
    assert torch.equal(y[:nan_at][~sees], clean[:nan_at, 0][~sees])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("n,first", [(64, 0), (150, 70), (6000, 0), (6000, 3333), (6000, 5936)])
def test_infinities_beside_a_nan_query(bqm, n, first, dt):
    # one token, four heads over one: the last one's query is NaN
    print("nan query", n, first, dt, file=sys.stderr, flush=True)
    s = Setup([n], [1], 1, 64, 16, dt, seed=41, n_q=4)
    _diagonal_infinities(s, first)
    s.q[0, 3] = NAN
    y = bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), s.batch(bqm))
    assert torch.isposinf(y[0, :3]).all()
    assert torch.isnan(y[0, 3]).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("n,q_len,group", [(90, 1, 4), (6000, 1, 4), (6000, 8, 4), (3000, 40, 1)])
def test_infinities_of_weights_near_zero(bqm, n, q_len, group, dt):
    # the last tokens' scores are 200 above the others': their weights are e^-200,
    # which is above zero, and an infinite value times that is infinite
    s = Setup([n], [q_len], 1, 64, 16, dt, seed=42, n_q=group)
    s.q.zero_()
    s.q[..., 0] = 16.0
    for j in range(n):
        s.k[int(s.table[0, j // 16]), j % 16, 0, 0] = 12.5 if j >= n - q_len - 3 else 0.0
    for j, d in ((5, 7), (n // 2, 20), (n // 2 + 1, 21)):
        s.v[int(s.table[0, j // 16]), j % 16, 0, d] = INF
    s.v[int(s.table[0, 9 // 16]), 9 % 16, 0, 30] = NAN
    y = bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), s.batch(bqm), scale=1.0).float()
    for d in (7, 20, 21):
        assert torch.isposinf(y[..., d]).all(), d
    assert torch.isnan(y[..., 30]).all()
    rest = [d for d in range(64) if d not in (7, 20, 21, 30)]
    assert torch.isfinite(y[..., rest]).all()


@pytest.mark.parametrize("out_dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens,q_lens,H,Hq,D", [
    ([50], [1], 1, 4, 64), ([3000], [1], 2, 8, 128), ([90], [90], 1, 2, 64), ([2900], [40], 1, 4, 40),
    ([700, 0, 33], [400, 1, 1], 1, 2, 128), ([300], [8], 1, 2, 256), ([2300], [2300], 8, 64, 128),
])
def test_values_near_the_largest_of_the_type(bqm, lens, q_lens, H, Hq, D, out_dt):
    # values up to 2^127 of either sign, sums of many of them above what 32 bits hold:
    # the weighted means are not
    print("large values", lens, q_lens, H, Hq, D, out_dt, file=sys.stderr, flush=True)
    s = Setup(lens, q_lens, H, D, 16, "bf16", seed=43, n_q=Hq)
    for b in range(len(lens)):
        # of one sign, so that sums of many go as high as they can
        s.vs[b] = (s.vs[b].abs().clamp(max=3.5) * 2.0 ** 125).to(DT["bf16"])
        s.store(s.v, b, s.vs[b])
    y = bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), s.batch(bqm), out_dtype=DT[out_dt])
    assert torch.isfinite(y.float()).all()
    if sum(q_lens) > 1000:  # rows 0, 97, 194, .. alone, the 64-bit form being slow
        keep = torch.arange(0, q_lens[0], 97, device="cuda")
        k, v = s.ks[0].double(), s.vs[0].double()
        for h in (0, 37, 63):
            x = (s.q[keep, h].double() @ k[:, h // 8].T.contiguous()) * D ** -0.5
            x.masked_fill_(torch.arange(lens[0], device="cuda")[None] > keep[:, None], -INF)
            want = torch.softmax(x, -1) @ v[:, h // 8].contiguous()
            err = (y[keep, h].double() - want).abs() / want
            # a weight's rounding to 8 bits above and one store; scores' rounding is far below
            assert float(err.max()) <= 3.0 * UNIT["bf16"]
    else:
        _close_attention(_f64(y), s, D ** -0.5, True, 0, out_dt)


@pytest.mark.parametrize("n,at,q_len,group,n_seqs,H", [
    (20000, 6000, 1, 4, 1, 1), (120000, 0, 1, 8, 1, 1), (20000, 9, 40, 1, 1, 1), (9000, 8000, 4, 2, 1, 1),
    (40000, 0, 40, 1, 64, 8), (20000, 100, 40, 4, 64, 2)])
def test_small_weights_of_many_tokens_in_16_bits(bqm, n, at, q_len, group, n_seqs, H):
    # one token whose value is 0 outweighs each of the others by e^18 (2^26): the
    # others' mean, times their share of the sum, is the output. (The sequences
    # share their pages; 64 of them fill the card without their tokens being cut.)
    print("small weights", n, at, q_len, group, n_seqs, H, file=sys.stderr, flush=True)
    s = Setup([n], [q_len], H, 64, 16, "f16", seed=44, n_q=group * H)
    for x in (s.k, s.v):
        x.zero_()
    q = torch.zeros(q_len * n_seqs, group * H, 64, dtype=DT["f16"], device="cuda")
    q[..., 0] = 4.0
    pages = torch.tensor(s.table[0, :-(-n // 16)]).cuda()
    s.v[pages] = 1000.0
    page, place = int(s.table[0, at // 16]), at % 16
    s.k[page, place, :, 0] = 4.5
    s.v[page, place] = 0.0
    batch = bqm.KvBatch(_ints(s.table.repeat(n_seqs, 0)), _ints([n] * n_seqs),
                        _ints([i * q_len for i in range(n_seqs + 1)]), max_q=q_len)
    y = bqm.paged_attention(q, bqm.KvCache(s.k, s.v), batch, scale=1.0, causal=False, out_dtype=torch.float32)
    e = math.exp(-18.0)
    want = 1000.0 * (n - 1) * e / (1.0 + (n - 1) * e)
    # a weight is kept to 2^-12 of itself or to 2^-32 of the row's largest; fp32 sums of
    # n terms and the exponential beside that
    bound = want * (2.0 ** -11 + n * 2.0 ** -24 + 2.0 ** -18) + 1000.0 * (n - 1) * 2.0 ** -32
    err = float((y.double() - want).abs().max())
    assert err <= bound, (err, want, bound)
