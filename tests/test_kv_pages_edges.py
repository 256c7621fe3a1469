"""Upkeep of the pages where its calls depend on order, and tables larger than one
segment of its masks, against the definition one page at a time."""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_attention import Model, _ints, _same, _state  # noqa: E402


@pytest.fixture(scope="module")
def bqm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_mat_amd as m
    m.library()
    return m


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("S,M,P,ps,seed", [(6, 8, 60, 4, 0), (60, 30, 900, 16, 1), (900, 40, 20000, 8, 2)])
def test_forks_of_children(bqm, S, M, P, ps, seed, in_place):
    # chains: each child is the parent of the next one. It held nothing before the
    # call, so only the first of a chain takes anything, in place too
    print("chains", S, M, P, ps, in_place, file=sys.stderr, flush=True)
    rng = np.random.default_rng(seed)
    table, lens, refs = _state(rng, S, M, P, ps)
    table[0], lens[0] = -1, 0
    # whole pages: what a chain's second fork would take without a page of its own
    full = lens // ps * ps
    for s in np.flatnonzero(lens % ps):
        p = table[s, lens[s] // ps]
        table[s, lens[s] // ps], refs[p] = -1, 0
    lens = full
    m = Model(table, lens, refs, ps)
    live, empty = np.flatnonzero(lens), np.flatnonzero(lens == 0)
    children = rng.permutation(empty)
    parents = np.concatenate(([live[0]], children[:-1]))
    again = rng.random(len(children)) < 0.3
    parents[again] = rng.choice(live, int(again.sum()))
    p = bqm.KvPages(_ints(m.t), _ints(m.l), _ints(m.r))
    q, moves, short = bqm.kv_fork(p, _ints(parents), _ints(children), ps, out=p if in_place else None)
    want, k = m.fork(parents, children)
    assert int(short) == k
    assert np.array_equal(moves.cpu().numpy(), np.array(want, int).reshape(-1, 3))
    _same(q, m)


def _around(edge, P, rng):
    """A state with used and free pages on both sides of page `edge`: rows of pages
    near it and anywhere, some free runs, no page shared."""
    S, M, ps = 40, 300, 16
    near = np.arange(max(0, edge - 2000), min(P, edge + 2000))
    rest = rng.permutation(np.setdiff1d(np.arange(P), near, assume_unique=True))
    pool = np.concatenate((rng.permutation(near), rest))
    table, lens, refs = np.full((S, M), -1), np.zeros(S, int), np.zeros(P, int)
    at = 0
    for s in range(S - 8):
        n = int(rng.integers(1, M * ps - 40))
        k = -(-n // ps)
        table[s, :k], lens[s] = pool[at:at + k], n
        refs[pool[at:at + k]] = 1
        at += k
    return table, lens, refs, ps


def _ranks(refs):
    """Free pages, lowest first."""
    return np.flatnonzero(refs <= 0)


class Wide(Model):
    """The same definition with the free pages found at once (the tables are long)."""

    def free_pages(self):
        return _ranks(self.r)

    def compact(self):
        n = int((self.r > 0).sum())
        at = np.arange(len(self.r))
        src, dst = at[(self.r > 0) & (at >= n)], at[(self.r <= 0) & (at < n)]
        to = at.copy()
        to[src] = dst
        self.r[dst], self.r[src] = self.r[src], 0
        self.t = np.where(self.t >= 0, to[np.maximum(self.t, 0)], self.t)
        moves = np.full((len(self.r) // 2, 3), (-1, -1, 0))
        moves[:len(src)] = np.stack((src, dst, np.full(len(src), self.ps)), 1)
        return moves, to


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("P", [262143, 262144, 262145, 600001])
def test_tables_of_several_segments(bqm, P, full, in_place):
    # the pages in use are kept as masks of 2^18 pages at a time; `full`: all pages
    # below the first segment's edge are held by one more count each, so that what is
    # given lies behind it
    print("segments", P, full, in_place, file=sys.stderr, flush=True)
    rng = np.random.default_rng(P)
    table, lens, refs, ps = _around(262144, P, rng)
    if full:
        refs[:min(P, 262144) - 5] += 1
    m = Wide(table, lens, refs, ps)
    p = bqm.KvPages(_ints(m.t), _ints(m.l), _ints(m.r))
    out = p if in_place else None
    for _ in range(2):
        n_new = rng.integers(0, 40, len(m.l))
        p, short = bqm.kv_extend(p, _ints(n_new), ps, out=out)
        assert int(short) == m.extend(n_new)
        _same(p, m)
        children = np.flatnonzero(m.l == 0)
        parents = rng.choice(np.flatnonzero(m.l > 0), len(children))
        p, moves, short = bqm.kv_fork(p, _ints(parents), _ints(children), ps, out=out)
        want, k = m.fork(parents, children)
        assert int(short) == k
        assert np.array_equal(moves.cpu().numpy(), np.array(want, int).reshape(-1, 3))
        _same(p, m)
        gone = [int(x) for x in rng.choice(len(m.l), 12, replace=False)]
        p = bqm.kv_free(p, _ints(gone), out=out)
        m.free(gone)
        _same(p, m)
        p, moves, to = bqm.kv_compact(p, ps, out=out)
        want, where = m.compact()
        assert np.array_equal(moves.cpu().numpy(), want)
        assert np.array_equal(to.cpu().numpy(), where)
        _same(p, m)
