"""The token side's two forms that keep sums in a workspace, rows of logits shared by several
workgroups and products cut into parts: repeated, captured and replayed, on two streams at once."""
import ctypes

import pytest
import torch

import bit_quantized_mat_amd as bqm
from bit_quantized_mat_amd.tokens import _Q4Struct

ROWS, LOGITS = 40, 80021
N, K, COLUMNS = 4096, 4096, 64


def test_these_sizes_are_shared_and_cut():
    lib = bqm.library()
    # a workspace for a few rows alone: sums of shared rows; one beyond the columns laid out: sums of parts
    assert lib.sample_workspace_bytes(ROWS, LOGITS) > lib.sample_workspace_bytes(ROWS - 1, LOGITS) > 0
    m = _Q4Struct(codes=None, scales=None, zeros=None, N=N, K=K, group=64)
    laid = COLUMNS // 32 * (K // 32) * (2048 + 128)
    assert lib.mm_q4_workspace_bytes(ctypes.byref(m), COLUMNS) >= laid + 3 * COLUMNS * N * 4


class Both:
    """A product in parts and a draw from shared rows."""

    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        codes = torch.randint(0, 256, (N, K // 2), generator=self.gen, device="cuda", dtype=torch.uint8)
        scales = (torch.rand(N, K // 64, generator=self.gen, device="cuda") * 0.02).half()
        self.m = bqm.Q4Matrix(codes, scales)
        self.x = torch.empty(COLUMNS, K, device="cuda")
        self.logits = torch.empty(ROWS, LOGITS, device="cuda")
        self.u = torch.empty(ROWS, device="cuda")
        self.settings = dict(top_k=torch.full((ROWS,), 300, device="cuda", dtype=torch.int32),
                             top_p=torch.full((ROWS,), 0.97, device="cuda"), min_p=torch.full((ROWS,), 1e-4, device="cuda"))
        self.new()

    def new(self):
        self.x.normal_(generator=self.gen)
        self.logits.normal_(generator=self.gen).mul_(3.0)
        self.u.uniform_(generator=self.gen)

    def run(self):
        y = bqm.mm_q4(self.m, bqm.q8_1_quantize(self.x))
        return (y, *bqm.sample(self.logits, self.u, **self.settings))


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
def test_repeated():
    b = Both(1)
    first = b.run()
    for _ in range(20):
        assert same(b.run(), first)


@pytest.mark.gpu
def test_captured():
    # two graphs of the same sizes, replayed in turn with new inputs, eager calls between the replays
    b = Both(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = b.run()
        graphs.append((g, out))
    for turn in range(8):
        b.new()
        g, out = graphs[turn % 2]
        g.replay()
        want = b.run()
        torch.cuda.synchronize()
        assert same(out, want), turn


@pytest.mark.gpu
def test_on_two_streams_at_once():
    both = [Both(3), Both(4)]
    want = [b.run() for b in both]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, b in enumerate(both):
            with torch.cuda.stream(streams[i]):
                got[i].append(b.run())
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert same(g, want[i])


@pytest.mark.gpu
def test_on_another_stream_than_the_current_one():
    b = Both(5)
    want = b.run()
    a = bqm.q8_1_quantize(b.x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        y = bqm.mm_q4(b.m, a, stream=s)
        t, lp = bqm.sample(b.logits, b.u, **b.settings, stream=s)
        s.synchronize()
        assert same((y, t, lp), want)
