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
