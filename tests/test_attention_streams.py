"""Calls of the attention side on a stream that is not the current one: their memory
is that stream's own, and they do not disturb calls still under way."""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_attention import Setup, _ints  # noqa: E402


@pytest.fixture(scope="module")
def bqm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_mat_amd as m
    m.library()
    return m


def _stream_of(t):
    """The stream whose memory the tensor's block was taken from."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment")


def _calls(bqm):
    """name -> call(stream): its new tensors."""
    s = Setup([40, 3000], [1, 1], 2, 64, 16, "bf16", seed=60, n_q=4, spare=9)
    cache, b = bqm.KvCache(s.k, s.v), s.batch(bqm, max_q=1)
    f = bqm.rope_inv_freq(64)
    table = bqm.rope_table(f, 3100)
    x = torch.randn(2, 8, 64, device="cuda")
    refs = np.zeros(s.k.shape[0], int)
    full = np.concatenate((s.table, np.full((1, s.table.shape[1]), -1)))
    refs[full[full >= 0]] = 1
    pages = bqm.KvPages(_ints(full), _ints([40, 3000, 0]), _ints(refs))
    one, two, gone, n_new = _ints([1]), _ints([2]), _ints([0]), _ints([9, 0, 0])
    flat = lambda r: [t for x in r for t in (x if isinstance(x, tuple) else (x,))]  # noqa: E731
    return {
        "rope_table": lambda st: [bqm.rope_table(f, 50, stream=st)],
        "rope": lambda st: [bqm.rope(x, table, _ints([3, 4]), stream=st)],
        "append": lambda st: [bqm.rope_kv_append(x[:, :4], x[:, 4:6], x[:, 6:], cache, b, table, stream=st)],
        "attention": lambda st: [bqm.paged_attention(s.q, cache, b, stream=st)],
        "extend": lambda st: flat(bqm.kv_extend(pages, n_new, 16, stream=st)),
        "fork": lambda st: flat(bqm.kv_fork(pages, one, two, 16, stream=st)),
        "free": lambda st: list(bqm.kv_free(pages, gone, stream=st)),
        "compact": lambda st: flat(bqm.kv_compact(pages, 16, stream=st)),
    }


def test_outputs_are_the_streams_own_memory(bqm):
    calls = _calls(bqm)
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    for name, call in calls.items():
        print("memory of", name, file=sys.stderr, flush=True)
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        got = call(side)
        torch.cuda.synchronize()
        assert torch.cuda.current_stream() == here
        for g, w in zip(got, want):
            assert torch.equal(g, w)
            assert _stream_of(g) == side.cuda_stream, name
        for t in call(None):
            assert _stream_of(t) == here.cuda_stream, name
        del got, g, t
        torch.cuda.synchronize()


@pytest.mark.parametrize("call", ["attention", "extend", "fork"])
def test_workspaces_are_the_streams_own_memory(bqm, call):
    # outputs given: what is left to allocate is the workspace
    s = Setup([6000], [1], 1, 64, 16, "bf16", seed=61, n_q=4)
    cache, b, out = bqm.KvCache(s.k, s.v), s.batch(bqm, max_q=1), torch.empty_like(s.q)
    pages = bqm.KvPages(_ints([[0, -1, -1], [-1, -1, -1]]), _ints([9, 0]), _ints([1, 0, 0, 0]))
    new = bqm.KvPages(*(torch.empty_like(t) for t in pages))
    n_new, one, two = _ints([1, 0]), _ints([0]), _ints([1])
    assert bqm.paged_attention_workspace_bytes(cache, b, 4, 1) > 0
    run = {"attention": lambda st: bqm.paged_attention(s.q, cache, b, out=out, stream=st),
           "extend": lambda st: bqm.kv_extend(pages, n_new, 16, out=new, stream=st),
           "fork": lambda st: bqm.kv_fork(pages, one, two, 16, out=new, stream=st)}[call]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    taken = {}
    for st in (None, side):
        torch.cuda.empty_cache()
        before = sum(x["allocated_size"] for x in torch.cuda.memory_snapshot() if x["stream"] == side.cuda_stream)
        torch.cuda.memory._record_memory_history(max_entries=1000)
        keep = run(st)
        trace = torch.cuda.memory._snapshot()["device_traces"][torch.cuda.current_device()]
        torch.cuda.memory._record_memory_history(enabled=None)
        torch.cuda.synchronize()
        taken[st] = {e["stream"] for e in trace if e["action"] == "alloc"}
        assert before == 0
        del keep
    assert taken[side] == {side.cuda_stream}
    assert taken[None] == {torch.cuda.current_stream().cuda_stream}


def test_calls_on_two_streams_overlap(bqm):
    # no synchronization between them: a long call cut into parts on the current
    # stream, whose workspace is given back when it returns, and at once others on
    # another stream
    a = Setup([20000] * 2, [1] * 2, 8, 128, 16, "bf16", seed=62, n_q=32)
    b = Setup([9000, 12000], [1] * 2, 8, 128, 16, "bf16", seed=63, n_q=32)
    runs = [(x.q, bqm.KvCache(x.k, x.v), x.batch(bqm, max_q=1)) for x in (a, b)]
    want = [bqm.paged_attention(*r) for r in runs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        got = []
        for _ in range(4):
            got.append((0, bqm.paged_attention(*runs[0])))
            got.append((1, bqm.paged_attention(*runs[1], stream=side)))
        torch.cuda.synchronize()
        for i, y in got:
            assert torch.equal(y, want[i])


def test_outputs_stay_until_the_current_stream_is_done(bqm):
    # an output of another stream, used on the current one and let go of: its memory
    # is not handed on before that use has run
    s = Setup([3000], [1], 2, 64, 16, "bf16", seed=64, n_q=4)
    cache, b = bqm.KvCache(s.k, s.v), s.batch(bqm, max_q=1)
    want = bqm.paged_attention(s.q, cache, b).float()
    other = torch.randn_like(s.q)
    big = torch.randn(4096, 4096, device="cuda")
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    y = bqm.paged_attention(s.q, cache, b, stream=side)
    here.wait_stream(side)
    for _ in range(20):
        big = torch.tanh(big @ big)
    got = y.float()  # behind all that
    done = here.record_event()
    at = y.data_ptr()
    del y
    later = [bqm.paged_attention(other, cache, b, stream=side) for _ in range(8)]
    if not done.query():
        assert all(t.data_ptr() != at for t in later)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_streams_of_other_kinds_are_refused(bqm):
    with pytest.raises((ValueError, AttributeError)):
        bqm.rope_table(bqm.rope_inv_freq(64), 4, stream=torch.Stream(device="cpu"))
