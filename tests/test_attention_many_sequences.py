"""Attention over batches of more sequences than a wave has lanes, and than the
pieces of few-row launches are counted for, single tokens and chunks, cut and not."""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_attention import DT, Setup, _close_attention, _f64, _ints  # noqa: E402


@pytest.fixture(scope="module")
def bqm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_mat_amd as m
    m.library()
    return m


def _ragged(n, seed, long, top):
    """n lengths: many short, some empty, a few of `long` tokens at both ends."""
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(top), n))]
    for b in (1, n // 2, n - 2):
        lens[b] = long + b
    for b in (0, n // 3, n - 1):
        lens[b] = 0
    return lens


@pytest.mark.parametrize("n", [64, 65, 127, 128, 129, 300, 4100])
@pytest.mark.parametrize("H,Hq,D,window", [(1, 4, 64, 0), (2, 2, 128, 300)])
def test_single_tokens(bqm, n, H, Hq, D, window):
    print("sequences", n, H, Hq, D, window, file=sys.stderr, flush=True)
    lens = _ragged(n, n, 5000, 60)
    s = Setup(lens, [1] * n, H, D, 16, "bf16", seed=n, n_q=Hq)
    out = torch.full(s.q.shape, float("nan"), dtype=DT["bf16"], device="cuda")
    b = s.batch(bqm, max_q=1, max_kv=max(lens))
    cache = bqm.KvCache(s.k, s.v)
    if n <= 300:
        assert window or bqm.paged_attention_workspace_bytes(cache, b, Hq, n) > 0  # cut
    y = bqm.paged_attention(s.q, cache, b, window=window, out=out)
    _close_attention(_f64(y), s, D ** -0.5, True, window)


@pytest.mark.parametrize("n", [65, 129, 300])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks_among_single_tokens(bqm, n, causal):
    # some sequences with no new token, two of many; more new tokens than tokens too
    rng = np.random.default_rng(n)
    lens = _ragged(n, n + 1, 900, 40)
    q_lens = [int(rng.choice([0, 1, 1, 1, 3])) for _ in range(n)]
    q_lens[2], q_lens[n - 3] = 70, 150
    lens[n - 3] = 200
    print("chunks", n, causal, file=sys.stderr, flush=True)
    s = Setup(lens, q_lens, 1, 64, 16, "f16", seed=n, n_q=2, order="head")
    out = torch.full(s.q.shape, float("nan"), dtype=DT["f16"], device="cuda")
    y = bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), s.batch(bqm), causal=causal, out=out)
    _close_attention(_f64(y), s, 0.125, causal, 0)


@pytest.mark.parametrize("n", [65, 200])
def test_drafts(bqm, n):
    # a few new tokens each, cut into parts
    lens = _ragged(n, n + 2, 4000, 50)
    q_lens = [min(4, max(1, x)) if x else 0 for x in lens]
    print("drafts", n, file=sys.stderr, flush=True)
    s = Setup(lens, q_lens, 2, 64, 24, "f16", seed=n, n_q=6)
    out = torch.full(s.q.shape, float("nan"), dtype=DT["f16"], device="cuda")
    y = bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), s.batch(bqm, max_q=4, max_kv=max(lens)), out=out)
    _close_attention(_f64(y), s, 0.125, True, 0)


@pytest.mark.parametrize("max_q", [1, 40])
def test_a_captured_call_replays_other_lengths(bqm, max_q):
    """One capture; then other lengths, rows and pages in the same arrays, within the
    bounds captured: each replay is what an eager call gives."""
    n, T, width, P, H, D, ps = 70, 70 if max_q == 1 else 400, 200, 3000, 2, 64, 16
    rng = np.random.default_rng(3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn(P, ps, H, D, device="cuda", generator=gen).half() for _ in range(2))
    q = torch.randn(T, 4, D, device="cuda", generator=gen).half()
    cache = bqm.KvCache(k, v)

    def lengths(i):
        if max_q == 1:
            q_lens = [1] * n
        else:
            cuts = np.sort(rng.integers(0, T + 1, n - 1))
            q_lens = np.minimum(np.diff(np.concatenate(([0], cuts, [T]))), max_q)
            short = T - int(q_lens.sum())
            for b in range(n):  # what the cap took off goes where there is room
                add = min(short, max_q - int(q_lens[b]))
                q_lens[b] += add
                short -= add
        kv = [int(x) for x in rng.integers(0, [40, 900, 60][i % 3], n)]
        for b in rng.integers(0, n, 3):
            kv[b] = int(rng.integers(2000, width * ps + 1))
        return _ints(kv), _ints(np.concatenate(([0], np.cumsum(q_lens)))), _ints(rng.integers(0, P, (n, width)))

    kv_lens, starts, table = (t.clone() for t in lengths(0))
    batch = bqm.KvBatch(table, kv_lens, starts, max_q=max_q)
    call = lambda: bqm.paged_attention(q, cache, batch)  # noqa: E731
    assert bqm.paged_attention_workspace_bytes(cache, batch, 4, T) > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call()
    seen = []
    for i in range(5):
        for to, new in zip((kv_lens, starts, table), lengths(i)):
            to.copy_(new)
        eager = call().clone()
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager), i
        seen.append(eager)
    assert not torch.equal(seen[0], seen[1])
