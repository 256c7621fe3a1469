"""The attention side on the GPU: rotary positions, the append into a paged
cache, attention over it and the upkeep of its pages, each against its
definition in 64 bits (numpy), at the sizes and masks where it can go wrong."""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# half a unit in the last place of a value in [1, 2): the rounding of one store
UNIT = {k: torch.finfo(d).eps / 2 for k, d in DT.items()}
# smallest spacing near zero (half of it is a store's absolute error there)
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def bqm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_mat_amd as m
    m.library()
    return m


def _f64(t):
    return t.detach().double().cpu().numpy()


def _ints(v):
    return torch.tensor(np.asarray(v, np.int32)).cuda()


# ---- rotary positions ----------------------------------------------------------

def _turn64(x, cs, interleaved, sign=1.0):
    """x [T, H, D] float64 by cs [T, F, 2]: (result, sum of |products| per value)."""
    f, y, mag = cs.shape[1], x.copy(), np.abs(x)
    c, s = cs[:, None, :, 0], sign * cs[:, None, :, 1]
    lo, hi = (slice(0, 2 * f, 2), slice(1, 2 * f, 2)) if interleaved else (slice(0, f), slice(f, 2 * f))
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    mag[..., lo], mag[..., hi] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return y, mag


def _close_turn(got, want, mag, dt):
    # two products and one sum in fp32 (three roundings), one store
    bound = 3.0 * 2.0 ** -24 * mag + 1.01 * UNIT[dt] * np.abs(want) + TINY[dt]
    assert np.all(np.abs(got - want) <= bound), float(np.max(np.abs(got - want) - bound))


@pytest.mark.parametrize("n_pos,n_rot,scale", [(1, 2, 1.0), (70, 64, 1.0), (1001, 128, 0.7)])
def test_rope_table(bqm, n_pos, n_rot, scale):
    f = bqm.rope_inv_freq(n_rot)
    t = _f64(bqm.rope_table(f, n_pos, scale=scale))
    a = np.arange(n_pos)[:, None] * _f64(f)
    want = scale * np.stack((np.cos(a), np.sin(a)), -1)
    # one rounding to fp32; sincos and the product in fp64 are off by far less
    assert np.all(np.abs(t - want) <= 2.0 ** -24 * np.abs(want) + 1e-12)


def test_rope_table_long_positions(bqm):
    # a position of two million: the angle is formed in fp64
    f = torch.tensor([1.0, 0.5, 1e-3], dtype=torch.float64, device="cuda")
    n = 2_000_001
    t = bqm.rope_table(f, n)[-1].double().cpu().numpy()
    a = (n - 1) * _f64(f)
    assert np.all(np.abs(t - np.stack((np.cos(a), np.sin(a)), -1)) <= 2.0 ** -24 + 1e-9)


def test_rope_inv_freq_scaling(bqm):
    f = bqm.rope_inv_freq(128, device="cpu")
    assert torch.equal(bqm.rope_inv_freq(128, factor=4.0, device="cpu"), f / 4)
    g = bqm.rope_inv_freq(128, factor=8.0, original=8192, low=1.0, high=4.0, device="cpu")
    turns = 8192 * f / (2 * np.pi)
    assert torch.equal(g[turns >= 4], f[turns >= 4]) and torch.equal(g[turns <= 1], f[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and ((g[mid] < f[mid]) & (g[mid] > f[mid] / 8)).all()


ROPE_CASES = [
    # T, H, D, F, interleaved, inverse
    (1, 1, 8, 4, False, False), (1, 32, 128, 64, False, False), (7, 3, 128, 64, True, True),
    (33, 5, 96, 48, False, True), (65, 2, 80, 20, True, False), (5, 4, 80, 20, False, False),
    (9, 7, 66, 16, False, False), (3, 2, 30, 7, True, False), (300, 8, 256, 32, False, False),
    (4, 1, 2, 1, True, True),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,H,D,F,inter,inverse", ROPE_CASES)
def test_rope(bqm, T, H, D, F, inter, inverse, dt):
    _say("rope", T, H, D, F, inter, inverse, dt)
    g = torch.Generator().manual_seed(T * 1000 + D)
    x = torch.randn(T, H, D, generator=g).to(DT[dt]).cuda()
    n_pos = 50
    table = bqm.rope_table(bqm.rope_inv_freq(2 * F), n_pos, scale=1.1)
    pos = torch.randint(-3, n_pos + 4, (T,), generator=g, dtype=torch.int32).cuda()  # clamped
    rows = _f64(table)[np.clip(pos.cpu().numpy(), 0, n_pos - 1)]
    want, mag = _turn64(_f64(x), rows, inter, -1.0 if inverse else 1.0)
    out = torch.full((T, H, D), float("nan"), dtype=DT[dt], device="cuda")
    y = bqm.rope(x, table, pos, interleaved=inter, inverse=inverse, out=out)
    _close_turn(_f64(y), want, mag, dt)
    # into 32 bits, from a strided view, and in place: the same values
    wide = torch.zeros(T, H + 2, D + 6, dtype=DT[dt], device="cuda")
    view = wide[:, 1:H + 1, 3:D + 3]
    view.copy_(x)
    _close_turn(_f64(bqm.rope(view, table, pos, interleaved=inter, inverse=inverse,
                              out_dtype=torch.float32)), want, mag, "f32")
    bqm.rope(view, table, pos, interleaved=inter, inverse=inverse, out=view)
    assert torch.equal(view, y)
    assert float(wide.double().abs().sum()) == float(view.double().abs().sum())  # nothing beside it


@pytest.mark.parametrize("inter", [False, True])
def test_rope_inverse_is_the_gradient(bqm, inter):
    T, H, D, F = 6, 2, 48, 16
    g = torch.Generator().manual_seed(3)
    x, w = (torch.randn(T, H, D, generator=g, dtype=torch.float64) for _ in range(2))
    table = bqm.rope_table(bqm.rope_inv_freq(2 * F), 40, scale=0.9)
    pos = _ints([0, 1, 5, 17, 30, 39])
    rows = _f64(table)[pos.cpu().numpy()]
    grad = bqm.rope(w.float().cuda(), table, pos, interleaved=inter, inverse=True)
    # the formula's gradient of sum(w * y) and differences of it, both in 64 bits
    want = np.zeros(x.shape)
    for i in np.ndindex(*x.shape):
        e = np.zeros(x.shape)
        e[i] = 1.0
        up = _turn64(x.numpy() + 0.5 * e, rows, inter)[0]
        down = _turn64(x.numpy() - 0.5 * e, rows, inter)[0]
        want[i] = np.sum(w.numpy() * (up - down))
    # linear: the difference is exact but for the cancellation of 64-bit sums;
    # w was rounded to fp32, then three fp32 roundings of at most 2 |w| scale
    assert np.max(np.abs(_f64(grad) - want)) <= 6 * 2.0 ** -24 * 2 * 0.9 * float(w.abs().max()) + 1e-9


# ---- cache helpers -----------------------------------------------------------------

class Setup:
    """A cache, a shuffled page table and the new tokens of some sequences."""

    def __init__(self, lens, q_lens, H, D, ps, dt, seed=0, order="token", spare=3, n_q=None,
                 fill=float("nan"), pages_wide=0):
        rng = np.random.default_rng(seed)
        self.lens, self.q_lens, self.H, self.D, self.ps, self.dt = lens, q_lens, H, D, ps, dt
        need = [-(-n // ps) for n in lens]
        P = sum(need) + spare
        perm = rng.permutation(P)
        width = max(need + [1]) + pages_wide
        self.table = np.full((len(lens), width), -1, np.int64)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        shape = (P, ps, H, D) if order == "token" else (P, H, ps, D)
        kv = []
        for _ in range(2):
            c = torch.full(shape, fill, dtype=DT[dt], device="cuda")
            kv.append(c if order == "token" else c.transpose(1, 2))
        self.k, self.v = kv
        self.starts = np.concatenate(([0], np.cumsum(q_lens)))
        self.n_q = n_q or H
        gen = torch.Generator().manual_seed(seed + 1)
        self.q = torch.randn(int(self.starts[-1]), self.n_q, D, generator=gen).to(DT[dt]).cuda()
        # every sequence's keys and values, as they stand in the cache
        self.ks, self.vs = [], []
        for b, n in enumerate(lens):
            for c, keep in ((self.k, self.ks), (self.v, self.vs)):
                x = torch.randn(n, H, D, generator=gen).to(DT[dt]).cuda()
                self.store(c, b, x)
                keep.append(x)

    def store(self, c, b, x, first=0):
        i = torch.arange(first, first + len(x))
        page = torch.tensor(self.table[b])[i // self.ps]
        c[page.cuda(), (i % self.ps).cuda()] = x

    def batch(self, bqm, **kw):
        return bqm.KvBatch(_ints(self.table), _ints(self.lens), _ints(self.starts), **kw)


def _attention64(s, scale, causal, window):
    """(result [total, heads, D], weighted mean of |v|, tokens seen) in 64 bits, from the tokens
    that each row sees alone."""
    q = _f64(s.q)
    out, mean = np.zeros(q.shape), np.zeros(q.shape)
    seen = np.zeros(q.shape[:2])
    spread = np.zeros(q.shape[:2])
    G = s.n_q // s.H
    for b, n in enumerate(s.lens):
        k, v = _f64(s.ks[b]), _f64(s.vs[b])
        for i in range(s.q_lens[b]):
            pos = n - s.q_lens[b] + i
            lo = max(0, pos - window + 1) if window else 0
            hi = min(n, pos + 1) if causal else n
            if hi <= lo:
                continue
            t = s.starts[b] + i
            for h in range(s.n_q):
                kk, vv = k[lo:hi, h // G], v[lo:hi, h // G]
                x = scale * (kk @ q[t, h])
                e = np.exp(x - x.max())
                out[t, h] = e @ vv / e.sum()
                mean[t, h] = e @ np.abs(vv) / e.sum()
                seen[t, h] = hi - lo
                spread[t, h] = scale * np.max(np.abs(kk) @ np.abs(q[t, h]))
    return out, mean, seen, spread


def _close_attention(got, s, scale, causal, window, out_dt=None):
    want, mean, seen, spread = _attention64(s, scale, causal, window)
    u, vmax = UNIT[s.dt], max([float(v.abs().max()) for v in s.vs if len(v)] + [0.0])
    # each weight is rounded to the cache's type (relative u in the numerator and
    # in the denominator; the weights' absolute spacing near zero for every token
    # seen); a score's fp32 sum of D products, its scaling and the exponential
    # move a weight by at most (D + 16) 2^-23 of the score's products and 2^-20;
    # fp32 accumulation over the tokens; one store
    rel = 2.0 * u + 2.0 * ((s.D + 16) * 2.0 ** -23 * spread + 2.0 ** -20) + seen * 2.0 ** -23
    bound = rel[..., None] * mean * 1.02 + UNIT[out_dt or s.dt] * np.abs(want) * 1.02
    bound += (2.0 * seen * TINY[s.dt] * vmax + TINY[out_dt or s.dt])[..., None]
    err = np.abs(got - want)
    assert np.all(err <= bound), (float(np.nanmax(err - bound)), int(np.isnan(err).sum()))
    assert np.all(got[seen == 0] == 0.0)


ATTN = [
    # lens, q_lens, heads, q heads, D, page, causal, window
    ([1], [1], 1, 1, 64, 16, True, 0),
    ([37], [1], 8, 32, 128, 16, True, 0),
    ([5, 0, 130, 17], [1, 1, 1, 1], 2, 8, 128, 16, True, 0),
    ([64, 65, 63, 128, 1], [1, 1, 1, 1, 1], 2, 4, 64, 64, True, 0),
    ([33], [33], 2, 2, 64, 16, True, 0),
    ([129], [129], 1, 4, 128, 24, True, 0),
    ([200, 70], [65, 70], 2, 14, 64, 32, True, 0),
    ([300], [40], 1, 1, 128, 1, True, 0),
    ([77, 3], [9, 3], 3, 3, 80, 7, True, 0),
    ([260, 90], [31, 2], 1, 8, 256, 16, True, 0),
    ([100], [100], 2, 2, 96, 100, True, 0),
    ([90, 20], [50, 7], 1, 5, 40, 48, True, 0),
    ([50], [13], 1, 3, 8, 5, True, 0),
    ([150], [20], 2, 4, 136, 16, True, 0),
    ([110], [6], 1, 2, 192, 16, False, 0),
    # sequences without new tokens, without tokens, with more new tokens than tokens
    ([40, 12, 0, 9, 3], [0, 4, 3, 0, 5], 2, 4, 64, 16, True, 0),
    # windows: shorter than a page, than a tile, than the sequence, and longer
    ([300], [300], 1, 2, 64, 16, True, 1),
    ([300, 41], [100, 41], 2, 4, 64, 16, True, 33),
    ([500], [1], 1, 8, 128, 16, True, 130),
    ([200], [150], 1, 1, 128, 32, True, 4000),
    # every token seen (an encoder's states): other lengths on both sides, and a window
    ([90, 1, 0], [7, 30, 2], 2, 4, 64, 16, False, 0),
    ([260], [70], 1, 2, 128, 16, False, 0),
    ([100], [40], 1, 2, 64, 16, False, 20),
    ([1700, 900], [1500, 12], 1, 2, 64, 16, False, 300),
    ([2000], [8], 1, 4, 64, 16, False, 100),
    ([2100, 700], [3, 5], 1, 2, 64, 16, True, 900),
    # one sequence far along a long axis, and rows that fill several tiles
    ([5000], [1], 1, 4, 128, 16, True, 0),
    ([3001], [3], 2, 4, 64, 16, True, 0),
    ([700], [400], 1, 2, 128, 64, True, 0),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lens,q_lens,H,Hq,D,ps,causal,window", ATTN)
def test_attention(bqm, lens, q_lens, H, Hq, D, ps, causal, window, dt):
    _say("attention", lens, q_lens, H, Hq, D, ps, causal, window, dt)
    # stale places hold NaN: none of it may come through
    s = Setup(lens, q_lens, H, D, ps, dt, seed=len(lens) + D, n_q=Hq, order="token" if D % 16 else "head",
              pages_wide=2)
    out = torch.full(s.q.shape, float("nan"), dtype=DT[dt], device="cuda")
    y = bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), s.batch(bqm), causal=causal, window=window,
                            out=out)
    _close_attention(_f64(y), s, D ** -0.5, causal, window)
    # closer bounds of the lengths, and 32 bits out
    b = s.batch(bqm, max_q=max(q_lens), max_kv=max(lens))
    y = bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), b, causal=causal, window=window,
                            out_dtype=torch.float32)
    _close_attention(_f64(y), s, D ** -0.5, causal, window, "f32")


@pytest.mark.parametrize("seed", range(12))
def test_attention_random(bqm, seed):
    rng = np.random.default_rng(100 + seed)
    n = int(rng.integers(1, 7))
    D = int(rng.choice([16, 48, 64, 72, 128, 160, 256]))
    H, G = int(rng.integers(1, 4)), int(rng.choice([1, 2, 3, 4, 6, 8, 16, 20]))
    top = int(rng.choice([1, 4, 40, 200]))
    q_lens = [int(rng.integers(0, top + 1)) for _ in range(n)]
    q_lens[0] = max(1, q_lens[0])
    lens = [int(x + rng.integers(0, 300)) for x in q_lens]
    ps, window = int(rng.choice([1, 6, 16, 33, 64])), int(rng.choice([0, 0, 1, 20, 150]))
    causal, dt = bool(rng.integers(0, 4)), str(rng.choice(["f16", "bf16"]))
    _say("attention random", seed, lens, q_lens, H, G, D, ps, window, causal, dt)
    s = Setup(lens, q_lens, H, D, ps, dt, seed=seed, n_q=H * G, order=str(rng.choice(["token", "head"])))
    y = bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), s.batch(bqm), scale=0.2, causal=causal,
                            window=window)
    _close_attention(_f64(y), s, 0.2, causal, window)


@pytest.mark.parametrize("lens,q_lens", [([150], [150]), ([90, 200], [3, 40]), ([70], [1])])
def test_attention_later_tokens_do_not_reach(bqm, lens, q_lens):
    # keys and values of the last new token are NaN and infinite: the rows
    # before it are as without it
    D = 64
    s = Setup(lens, q_lens, 2, D, 16, "f16", seed=5, n_q=4)
    cache = bqm.KvCache(s.k, s.v)
    clean = bqm.paged_attention(s.q, cache, s.batch(bqm))
    for b in range(len(lens)):
        for c, x in ((s.k, float("nan")), (s.v, float("inf"))):
            s.store(c, b, torch.full((1, 2, D), x, dtype=DT["f16"], device="cuda"), lens[b] - 1)
    dirty = bqm.paged_attention(s.q, cache, s.batch(bqm))
    last = torch.tensor(s.starts[1:] - 1)
    keep = torch.ones(len(s.q), dtype=torch.bool)
    keep[last] = False
    assert torch.equal(clean[keep.cuda()], dirty[keep.cuda()])
    assert torch.isnan(dirty[last.cuda()]).all()


@pytest.mark.parametrize("lens,q_lens,window", [([150], [150], 20), ([400], [30], 50)])
def test_attention_tokens_before_the_window_do_not_reach(bqm, lens, q_lens, window):
    D = 128
    s = Setup(lens, q_lens, 1, D, 16, "bf16", seed=6, n_q=2)
    cache = bqm.KvCache(s.k, s.v)
    clean = bqm.paged_attention(s.q, cache, s.batch(bqm), window=window)
    first = lens[0] - q_lens[0]  # the first row's place
    for c in (s.k, s.v):
        s.store(c, 0, torch.full((first + 1, 1, D), float("inf"), dtype=DT["bf16"], device="cuda"))
    dirty = bqm.paged_attention(s.q, cache, s.batch(bqm), window=window)
    assert torch.equal(clean[window:], dirty[window:])
    assert not torch.isfinite(dirty[:window].float()).any()


@pytest.mark.parametrize("dt,size", [("f16", 60.0), ("bf16", 300.0)])
def test_attention_large_scores(bqm, dt, size):
    # scores of tens of thousands: the maximum is taken before the exponential
    s = Setup([130, 300], [5, 1], 1, 64, 16, dt, seed=8, n_q=2)
    s.q *= size
    y = bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), s.batch(bqm), scale=1.0)
    _close_attention(_f64(y), s, 1.0, True, 0)


def test_attention_strided_queries_and_other_stream(bqm):
    s = Setup([70, 200], [3, 64], 2, 64, 16, "bf16", seed=9, n_q=4)
    cache, b = bqm.KvCache(s.k, s.v), s.batch(bqm)
    want = bqm.paged_attention(s.q, cache, b)
    rows = torch.full((len(s.q), 8, 80), float("nan"), dtype=DT["bf16"], device="cuda")
    view = rows[:, 2:6, 8:72]
    view.copy_(s.q)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    outs = [bqm.paged_attention(view, cache, b, stream=stream) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_attention_pages_of_nobody(bqm):
    # a place of the table without a page reads as zeros
    s = Setup([40], [1], 1, 64, 16, "f16", seed=10, fill=0.0)
    s.table[0, 1] = -1
    s.ks[0][16:32] = 0
    s.vs[0][16:32] = 0
    y = bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), s.batch(bqm))
    _close_attention(_f64(y), s, 0.125, True, 0)


def test_attention_far_pages(bqm):
    # a cache whose offsets pass 32 bits, in elements and in 16-byte pieces' bytes
    D, H, ps, P = 128, 2, 64, 150_000  # 2.46e9 elements, 4.9 GB each
    s = Setup([100, 300], [1, 20], H, D, ps, "bf16", seed=11, n_q=4)
    n = int(s.table.max()) + 1
    k, v = (torch.empty(P, ps, H, D, dtype=DT["bf16"], device="cuda") for _ in range(2))
    k[P - n:], v[P - n:] = s.k[:n], s.v[:n]
    b = bqm.KvBatch(_ints(np.where(s.table >= 0, s.table + P - n, -1)), _ints(s.lens), _ints(s.starts))
    assert torch.equal(bqm.paged_attention(s.q, bqm.KvCache(k, v), b),
                       bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), s.batch(bqm)))


def test_attention_pages_just_below_4_gib(bqm):
    # the last places that 32-bit offsets of bytes reach, and heads shorter than a tile
    D, H, ps = 80, 2, 64
    P = 0xfffff000 // (ps * H * D * 2)
    s = Setup([100, 300], [1, 20], H, D, ps, "f16", seed=13, n_q=4)
    n = int(s.table.max()) + 1
    k, v = (torch.empty(P, ps, H, D, dtype=DT["f16"], device="cuda") for _ in range(2))
    k[P - n:], v[P - n:] = s.k[:n], s.v[:n]
    b = bqm.KvBatch(_ints(np.where(s.table >= 0, s.table + P - n, -1)), _ints(s.lens), _ints(s.starts))
    assert torch.equal(bqm.paged_attention(s.q, bqm.KvCache(k, v), b),
                       bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), s.batch(bqm)))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lens,q_lens,H,Hq,D,ps,causal,window", [
    # rows that fill tiles, their tokens cut into parts, uneven ones and one of a few tokens
    ([2900], [40], 1, 4, 40, 16, True, 0),
    ([1500, 0, 700, 2111], [50, 0, 3, 33], 2, 4, 64, 24, True, 0),
    ([2500, 900], [130, 60], 1, 3, 64, 16, True, 1700),
    ([1801, 40], [33, 40], 1, 4, 128, 16, True, 0),
    ([1400], [200], 2, 2, 96, 7, False, 0),
    ([1290], [35], 1, 2, 136, 16, True, 0),
])
def test_attention_parts_of_many_rows(bqm, lens, q_lens, H, Hq, D, ps, causal, window, dt):
    _say("attention parts", lens, q_lens, H, Hq, D, ps, causal, window, dt)
    s = Setup(lens, q_lens, H, D, ps, dt, seed=D + len(lens), n_q=Hq)
    y = bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), s.batch(bqm), causal=causal, window=window)
    _close_attention(_f64(y), s, D ** -0.5, causal, window)
    b = s.batch(bqm, max_q=max(q_lens), max_kv=max(lens))
    y = bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), b, causal=causal, window=window,
                            out_dtype=torch.float32)
    _close_attention(_f64(y), s, D ** -0.5, causal, window, "f32")


def test_attention_is_repeatable(bqm):
    s = Setup([4000, 900, 33], [1, 17, 33], 2, 128, 16, "bf16", seed=12, n_q=8)
    cache, b = bqm.KvCache(s.k, s.v), s.batch(bqm)
    first = bqm.paged_attention(s.q, cache, b)
    for _ in range(5):
        assert torch.equal(bqm.paged_attention(s.q, cache, b), first)


# ---- append --------------------------------------------------------------------------

@pytest.mark.parametrize("src,dt", [("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("lens,q_lens,H,Hq,D,F,ps,inter,order", [
    ([9], [1], 2, 8, 128, 64, 16, False, "token"),
    ([40, 5, 3, 0], [17, 0, 3, 0], 1, 3, 64, 16, 16, True, "head"),
    ([31, 2], [5, 4], 2, 2, 72, 10, 7, False, "token"),   # more new tokens than tokens
    ([300], [300], 2, 4, 96, 48, 24, False, "head"),
])
def test_rope_kv_append(bqm, lens, q_lens, H, Hq, D, F, ps, inter, order, src, dt):
    _say("append", lens, q_lens, H, Hq, D, F, ps, inter, order, src, dt)
    s = Setup(lens, q_lens, H, D, ps, dt, seed=20, order=order, fill=7.0)
    T = int(s.starts[-1])
    gen = torch.Generator().manual_seed(21)
    row = torch.randn(T, Hq + 2 * H, D, generator=gen).to(DT[src]).cuda()
    q, k, v = row[:, :Hq], row[:, Hq:Hq + H], row[:, Hq + H:]
    table = bqm.rope_table(bqm.rope_inv_freq(2 * F), 400)
    before = (s.k.clone(), s.v.clone())
    q_out = torch.full((T, Hq, D), float("nan"), dtype=DT[dt], device="cuda")
    bqm.rope_kv_append(q, k, v, bqm.KvCache(s.k, s.v), s.batch(bqm), table, interleaved=inter,
                       q_out=q_out)
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, q_lens)]).astype(int)
    cs = _f64(table)[np.clip(pos, 0, 399)]
    _close_turn(_f64(q_out), *_turn64(_f64(q), cs, inter), dt)
    kk, mag = _turn64(_f64(k), cs, inter)
    seq = np.repeat(np.arange(len(lens)), q_lens)
    untouched = torch.ones(s.k.shape[:2], dtype=torch.bool)
    for t in range(T):
        if pos[t] < 0:
            continue
        page, at = s.table[seq[t], pos[t] // ps], pos[t] % ps
        _close_turn(_f64(s.k[page, at])[None], kk[t][None], mag[t][None], dt)
        assert torch.equal(s.v[page, at], v[t].to(DT[dt]))
        untouched[page, at] = False
    u = untouched.cuda()
    assert torch.equal(s.k[u], before[0][u]) and torch.equal(s.v[u], before[1][u])
    # positions of the caller's own, and keys and values alone
    own = _ints(np.clip(pos, 0, 390) + 3)
    s.k.copy_(before[0])
    bqm.rope_kv_append(None, k, v, bqm.KvCache(s.k, s.v), s.batch(bqm), table, positions=own,
                       interleaved=inter)
    kk, mag = _turn64(_f64(k), _f64(table)[own.cpu().numpy()], inter)
    for t in range(T):
        if pos[t] >= 0:
            _close_turn(_f64(s.k[s.table[seq[t], pos[t] // ps], pos[t] % ps])[None], kk[t][None],
                        mag[t][None], dt)


def test_append_skips_tokens_without_a_page(bqm):
    s = Setup([20], [20], 1, 64, 16, "f16", seed=22, fill=1.0)
    s.table[0, 1] = -1
    s.k.fill_(1.0)
    x = torch.zeros(20, 1, 64, device="cuda")
    bqm.rope_kv_append(None, x, x, bqm.KvCache(s.k, s.v), s.batch(bqm),
                       bqm.rope_table(bqm.rope_inv_freq(64), 32))
    assert int((s.k == 0).sum()) == 16 * 64


# ---- pages ---------------------------------------------------------------------------

class Model:
    """The page upkeep by its definition, one page at a time."""

    def __init__(self, table, lens, refs, ps):
        self.t, self.l, self.r, self.ps = table.copy(), lens.copy(), refs.copy(), ps

    def free_pages(self):
        return [p for p, r in enumerate(self.r) if r <= 0]

    def extend(self, n_new):
        free, rank, short, ps = self.free_pages(), 0, 0, self.ps
        lens = self.l.copy()
        for s, n in enumerate(n_new):
            have, want = -(-self.l[s] // ps), -(-(self.l[s] + max(n, 0)) // ps)
            if n > 0 and want > self.t.shape[1]:
                short += 1
                continue
            rank += want - have
            if want > have and rank > len(free):
                short += 1
                continue
            for j in range(have, want):
                p = free[rank - want + j]
                self.t[s, j], self.r[p] = p, 1
            lens[s] += max(n, 0)
        self.l = lens
        return short

    def fork(self, parents, children):
        free, rank, short, moves = self.free_pages(), 0, 0, []
        t, l, ps = self.t.copy(), self.l.copy(), self.ps
        for a, c in zip(parents, children):
            if not (0 <= a < len(l) and 0 <= c < len(l)):
                moves.append((-1, -1, 0))
                continue
            n = l[a]
            row = np.full(t.shape[1], -1)
            move = (-1, -1, 0)
            if n % ps:
                rank += 1
                if rank > len(free):
                    short += 1
                    n = 0
                else:
                    p = free[rank - 1]
                    move = (t[a, n // ps], p, n % ps)
                    row[n // ps], self.r[p] = p, 1
            row[:n // ps] = t[a, :n // ps]
            for p in row[:n // ps]:
                self.r[p] += 1
            self.t[c], self.l[c] = row, n
            moves.append(move)
        return moves, short

    def free(self, seqs):
        for s in set(seqs):
            if 0 <= s < len(self.l):
                for p in self.t[s]:
                    if p >= 0:
                        self.r[p] -= 1
                self.t[s], self.l[s] = -1, 0

    def compact(self):
        n = int((self.r > 0).sum())
        src = [p for p in range(n, len(self.r)) if self.r[p] > 0]
        dst = [p for p in range(n) if self.r[p] <= 0]
        to = np.arange(len(self.r))
        for a, b in zip(src, dst):
            to[a], self.r[b], self.r[a] = b, self.r[a], 0
        self.t = np.where(self.t >= 0, to[np.maximum(self.t, 0)], self.t)
        moves = [(a, b, self.ps) for a, b in zip(src, dst)]
        return moves + [(-1, -1, 0)] * (len(self.r) // 2 - len(moves)), to


def _state(rng, S, M, P, ps, full=0.6):
    """Sequences over random pages: some rows empty, no page shared."""
    table, lens, refs = np.full((S, M), -1), np.zeros(S, int), np.zeros(P, int)
    perm, at = rng.permutation(P), 0
    for s in range(S):
        n = int(rng.integers(0, M * ps + 1)) if rng.random() < full else 0
        n = min(n, (int(P * 0.7) - at) * ps)
        k = -(-n // ps)
        table[s, :k], lens[s] = perm[at:at + k], n
        refs[perm[at:at + k]] = 1
        at += k
    return table, lens, refs


def _same(p, m):
    assert np.array_equal(p.lens.cpu().numpy(), m.l)
    assert np.array_equal(p.table.cpu().numpy(), m.t)
    assert np.array_equal(p.refs.cpu().numpy(), m.r)


PAGES = [(1, 1, 1, 4, 0), (5, 7, 40, 16, 1), (64, 30, 900, 16, 2), (9, 3, 11, 1, 3),
         (300, 200, 30000, 24, 4), (1500, 17, 20011, 5, 5), (40, 700, 9000, 64, 6)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("S,M,P,ps,seed", PAGES)
def test_pages(bqm, S, M, P, ps, seed, in_place):
    _say("pages", S, M, P, ps, seed, in_place)
    rng = np.random.default_rng(seed)
    m = Model(*_state(rng, S, M, P, ps), ps)
    p = bqm.KvPages(_ints(m.t), _ints(m.l), _ints(m.r))
    out = p if in_place else None
    for step in range(4):
        n_new = np.where(rng.random(S) < 0.5, rng.integers(-1, 3 * ps, S), 0)
        p, short = bqm.kv_extend(p, _ints(n_new), ps, out=out)
        assert int(short) == m.extend(n_new)
        _same(p, m)
        empty = [s for s in range(S) if m.l[s] == 0]
        children = rng.permutation(empty)[:max(0, len(empty) - step)].astype(int)
        parents = rng.integers(0, S, len(children))
        parents = np.where(np.isin(parents, children), -5, parents)  # a child is no parent: left out
        p, moves, short = bqm.kv_fork(p, _ints(parents), _ints(children), ps, out=out)
        want, k = m.fork(parents, children)
        assert int(short) == k
        assert np.array_equal(moves.cpu().numpy(), np.array(want, int).reshape(-1, 3))
        _same(p, m)
        gone = list(rng.integers(-2, S + 2, max(1, S // 3)))  # some twice, some outside
        p = bqm.kv_free(p, _ints(gone), out=out)
        m.free(gone)
        _same(p, m)
        p, moves, to = bqm.kv_compact(p, ps, out=out)
        want, where = m.compact()
        assert np.array_equal(moves.cpu().numpy(), np.array(want, int).reshape(-1, 3))
        assert np.array_equal(to.cpu().numpy(), where)
        _same(p, m)


def test_pages_run_out(bqm):
    # 4 free pages: the first two sequences take three, the third wants two, the
    # fourth needs none, the fifth would fit but comes after
    ps, table = 4, np.full((5, 6), -1)
    table[:, 0] = np.arange(5)
    lens, refs = np.array([4, 3, 4, 1, 4]), np.array([1] * 5 + [0] * 4)
    m = Model(table, lens, refs, ps)
    p = bqm.KvPages(_ints(table), _ints(lens), _ints(refs))
    n_new = np.array([8, 2, 8, 2, 1])
    q, short = bqm.kv_extend(p, _ints(n_new), ps)
    assert int(short) == m.extend(n_new) == 2
    _same(q, m)
    # forks: two partly filled parents and one free page
    m = Model(np.array([[0, 1], [2, -1], [-1, -1], [-1, -1]]), np.array([7, 4, 0, 0]),
              np.array([1, 1, 1, 0]), ps)
    p = bqm.KvPages(_ints(m.t), _ints(m.l), _ints(m.r))
    q, moves, short = bqm.kv_fork(p, _ints([0, 0]), _ints([2, 3]), ps)
    want, k = m.fork([0, 0], [2, 3])
    assert int(short) == k == 1 and moves.cpu().tolist() == [list(x) for x in want]
    _same(q, m)


def test_extend_refuses_rows_past_the_table(bqm):
    p = bqm.KvPages(_ints([[0, -1], [1, -1]]), _ints([4, 4]), _ints([1, 1, 0, 0, 0]))
    q, short = bqm.kv_extend(p, _ints([9, 4]), 4)
    assert int(short) == 1 and q.lens.cpu().tolist() == [4, 8]
    assert q.table.cpu().tolist() == [[0, -1], [1, 2]] and q.refs.cpu().tolist() == [1, 1, 1, 0, 0]
    q, short = bqm.kv_extend(p, _ints([2 ** 31 - 1, 0]), 4)
    assert int(short) == 1 and q.lens.cpu().tolist() == [4, 4]


@pytest.mark.parametrize("L,P,ps,H,D,order", [(1, 9, 16, 2, 64, "token"), (3, 40, 24, 3, 40, "head"),
                                              (2, 300, 64, 8, 128, "token"), (1, 5, 1, 1, 8, "token")])
def test_copy_pages(bqm, L, P, ps, H, D, order):
    rng = np.random.default_rng(P)
    shape = (L, P, ps, H, D) if order == "token" else (L, P, H, ps, D)
    k, v = (torch.randn(shape, device="cuda").half() for _ in range(2))
    if order == "head":
        k, v = k.transpose(2, 3), v.transpose(2, 3)
    perm = rng.permutation(P)
    n = P // 2
    moves = [(perm[i], perm[n + i], int(rng.integers(0, ps + 1))) for i in range(n)]
    moves[0] = (perm[0], perm[n], ps + 100)  # at most a page
    moves += [(-1, -1, 0), (0, P, ps), (P, 0, ps)]
    wk, wv = k.clone(), v.clone()
    for a, b, t in moves[:n]:
        wk[:, b, :t], wv[:, b, :t] = wk[:, a, :t], wv[:, a, :t]
    bqm.kv_copy_pages(bqm.KvCache(k, v), _ints(moves))
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_empty_calls(bqm):
    s = Setup([5], [0], 1, 64, 16, "f16")
    cache, b = bqm.KvCache(s.k, s.v), s.batch(bqm)
    table = bqm.rope_table(bqm.rope_inv_freq(64), 8)
    assert bqm.paged_attention(s.q, cache, b).shape == (0, 1, 64)
    bqm.rope_kv_append(None, s.q, s.q, cache, b, table)
    bqm.rope(s.q, table, _ints([]))
    p = bqm.KvPages(_ints([[0, 1]]), _ints([5]), _ints([1, 1]))
    none = _ints([])
    q, moves, short = bqm.kv_fork(p, none, none, 4)
    assert q.table.cpu().tolist() == [[0, 1]] and moves.shape == (0, 3) and int(short) == 0
    bqm.kv_copy_pages(cache, moves)
    assert bqm.kv_free(p, none).lens.cpu().tolist() == [5]


def test_graph_replays(bqm):
    """A decode step (extend, append, attend, fork, copy, free, compact) in one graph."""
    D, H, Hq, ps = 64, 2, 4, 16
    s = Setup([40, 2000, 7], [1, 1, 1], H, D, ps, "bf16", seed=30, n_q=Hq, spare=9, fill=0.0, pages_wide=3)
    S = 4
    table = np.concatenate((s.table, np.full((1, s.table.shape[1]), -1)))
    refs = np.zeros(s.k.shape[0], int)
    refs[table[table >= 0]] = 1
    pages = bqm.KvPages(_ints(table), _ints([39, 1999, 6, 0]), _ints(refs))
    cache, angles = bqm.KvCache(s.k, s.v), bqm.rope_table(bqm.rope_inv_freq(D), 2100)
    x = torch.randn(3, Hq + 2 * H, D, device="cuda")
    n_new, starts = _ints([1, 1, 1, 0]), _ints([0, 1, 2, 3, 3])
    one, three, gone = _ints([1]), _ints([3]), _ints([0])

    def step():
        p, _ = bqm.kv_extend(pages, n_new, ps)
        b = bqm.KvBatch(p.table, p.lens, starts, max_q=1)
        q = bqm.rope_kv_append(x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], cache, b, angles)
        y = bqm.paged_attention(q, cache, b)
        p, moves, _ = bqm.kv_fork(p, one, three, ps)
        bqm.kv_copy_pages(cache, moves)
        p = bqm.kv_free(p, gone)
        p, moves, where = bqm.kv_compact(p, ps)
        return (q, y, where, moves) + tuple(p)

    keep = (s.k.clone(), s.v.clone())
    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for rep in range(4):
        s.k.copy_(keep[0])
        s.v.copy_(keep[1])
        for t in outs:
            t.view(torch.uint8).fill_(0xA5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (t, e) in enumerate(zip(outs, eager)):
            assert torch.equal(t, e), (rep, i)


def test_binding_refuses(bqm):
    s = Setup([20], [2], 2, 64, 16, "f16", seed=31, n_q=4)
    cache, b = bqm.KvCache(s.k, s.v), s.batch(bqm)
    table = bqm.rope_table(bqm.rope_inv_freq(64), 32)
    with pytest.raises(TypeError):
        bqm.KvCache(s.k.float(), s.v.float())
    with pytest.raises(ValueError):
        bqm.KvCache(s.k, s.v[:, :, :1])
    with pytest.raises(ValueError):
        bqm.KvCache(s.k.transpose(-1, -2), s.v.transpose(-1, -2))
    with pytest.raises(TypeError):
        bqm.paged_attention(s.q.float(), cache, b)
    with pytest.raises(TypeError):
        bqm.paged_attention(s.q.cpu(), cache, b)
    with pytest.raises(ValueError):
        bqm.paged_attention(s.q[:, :, :32], cache, b)
    with pytest.raises(bqm.BqmError):
        bqm.paged_attention(s.q[:, :3], cache, b)                      # 3 heads over 2
    with pytest.raises(bqm.BqmError):
        bqm.paged_attention(s.q, cache, b, scale=0.0)
    with pytest.raises(bqm.BqmError):
        bqm.paged_attention(s.q, cache, b, window=-1)
    with pytest.raises(ValueError):
        bqm.paged_attention(s.q, cache, b, out=torch.empty(2, 4, 32, device="cuda").half())
    with pytest.raises(TypeError):
        bqm.KvBatch(_ints(s.table).long(), _ints(s.lens), _ints(s.starts))
    with pytest.raises(ValueError):
        bqm.KvBatch(_ints(s.table), _ints(s.lens), _ints(s.starts)[1:])
    k = torch.zeros(2, 2, 64, device="cuda")
    with pytest.raises(ValueError):
        bqm.rope_kv_append(None, k[:, :1], k[:, :1], cache, b, table)
    with pytest.raises(ValueError):
        bqm.rope_kv_append(None, k, torch.zeros(2, 2, 128, device="cuda")[:, :, ::2], cache, b, table)
    with pytest.raises(bqm.BqmError):
        bqm.rope(k, bqm.rope_table(bqm.rope_inv_freq(130), 4), _ints([0, 1]))
    with pytest.raises(ValueError):
        bqm.rope(k, table, _ints([0]))
    p = bqm.KvPages(_ints([[0, 1]]), _ints([5]), _ints([1, 1]))
    with pytest.raises(ValueError):
        bqm.kv_free(p, _ints([0]), out=bqm.KvPages(_ints([[0]]), _ints([5]), _ints([1, 1])))
    with pytest.raises(bqm.BqmError):
        bqm.kv_extend(p, _ints([1]), 0)
    with pytest.raises(ValueError):
        bqm.kv_copy_pages(cache, _ints([[1, 2]]))


# Calls of many rows, whose tiles are the widest: every fourth row or so against the
# definition in 64 bits (on the GPU: the same formulas, torch's float64).

def _rows64(s, b, rows, h, scale, causal, window):
    k, v = (x[b][:, h // (s.n_q // s.H)].double() for x in (s.ks, s.vs))
    n = s.lens[b]
    q = s.q[s.starts[b] + rows, h].double()
    x = scale * (q @ k.T.contiguous())
    j, pos = torch.arange(n, device="cuda")[None], (n - s.q_lens[b] + rows)[:, None]
    hide = torch.zeros_like(x, dtype=torch.bool)
    if causal:
        hide |= j > pos
    if window:
        hide |= j <= pos - window
    p = torch.softmax(x.masked_fill(hide, float("-inf")), -1)
    spread = scale * (q.abs() @ k.abs().T.contiguous()).amax(-1)
    return p @ v, p @ v.abs(), (~hide).sum(-1), spread


@pytest.mark.parametrize("lens,q_lens,H,Hq,D,ps,causal,window,dt", [
    ([4133], [4133], 8, 32, 128, 16, True, 0, "bf16"),
    ([2500, 1900, 700], [2477, 1900, 31], 8, 32, 64, 24, True, 0, "f16"),
    ([3000, 2111], [2600, 2111], 8, 32, 128, 64, True, 700, "f16"),
    ([2300, 65, 2000], [2300, 65, 2000], 8, 56, 80, 16, True, 0, "bf16"),
    ([600, 64], [4100, 300], 8, 32, 128, 16, False, 0, "bf16"),
    ([4200, 900], [4100, 700], 8, 32, 64, 16, False, 500, "bf16"),
])
def test_attention_many_rows(bqm, lens, q_lens, H, Hq, D, ps, causal, window, dt):
    _say("attention many rows", lens, q_lens, H, Hq, D, ps, causal, window, dt)
    s = Setup(lens, q_lens, H, D, ps, dt, seed=D, n_q=Hq)
    scale = D ** -0.5
    out = torch.full(s.q.shape, float("nan"), dtype=DT[dt], device="cuda")
    y = bqm.paged_attention(s.q, bqm.KvCache(s.k, s.v), s.batch(bqm), causal=causal, window=window, out=out)
    assert torch.isfinite(y.float()).all()
    u, vmax = UNIT[dt], max(float(v.abs().max()) for v in s.vs)
    for b in range(len(lens)):
        rows = torch.unique(torch.cat((torch.arange(0, q_lens[b], 3), torch.tensor([q_lens[b] - 1])))).cuda()
        for h in range(0, Hq, 5):
            want, mean, seen, spread = _rows64(s, b, rows, h, scale, causal, window)
            rel = 2.0 * u + 2.0 * ((D + 16) * 2.0 ** -23 * spread + 2.0 ** -20) + seen * 2.0 ** -23
            bound = rel[:, None] * mean * 1.02 + u * want.abs() * 1.02
            bound += (2.0 * seen * TINY[dt] * vmax + TINY[dt])[:, None]
            err = (y[s.starts[b] + rows, h].double() - want).abs()
            assert (err <= bound).all(), (b, h, float((err - bound).max()))


def test_attention_many_rows_infinities_and_nan(bqm):
    # one infinite value and one NaN, in one head: only rows that see them change,
    # and those get them
    s = Setup([4200], [4200], 8, 128, 16, "bf16", seed=77, n_q=32)
    cache = bqm.KvCache(s.k, s.v)
    clean = bqm.paged_attention(s.q, cache, s.batch(bqm))
    for token, head, d, x in ((1000, 2, 5, float("inf")), (1700, 2, 99, float("nan"))):
        s.v[int(s.table[0, token // 16]), token % 16, head, d] = x
    y = bqm.paged_attention(s.q, cache, s.batch(bqm))
    mask = torch.zeros(y.shape, dtype=torch.bool, device="cuda")
    mask[1000:, 8:12, 5] = True
    mask[1700:, 8:12, 99] = True
    assert torch.equal(y[~mask], clean[~mask])
    assert torch.isposinf(y[1000:, 8:12, 5].float()).all()
    assert torch.isnan(y[1700:, 8:12, 99].float()).all()
