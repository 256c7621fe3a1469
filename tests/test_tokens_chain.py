"""The token side on the GPU as it is used: one operator after another, captured and
replayed, on other streams, beside one another."""
import math

import pytest
import torch

import bit_quantized_mat_amd as bqm

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


class Ends:
    """A table and an output matrix in 4 bits around one ternary product: token in, token out."""

    def __init__(self, vocab=1003, dim=512, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.dim = vocab, dim
        self.table = bqm.q4_quantize(torch.randn(vocab, dim, generator=g, device="cuda"), group=32)
        self.head = bqm.q4_quantize(torch.randn(vocab, dim, generator=g, device="cuda") / 8, group=128, zeros=True)
        trits = torch.randint(-1, 2, (dim, dim), generator=g, device="cuda", dtype=torch.int8)
        self.w = bqm.tq1_pack(trits, torch.full((dim, dim // 256), 0.05, device="cuda", dtype=torch.float16))
        self.gain = 1.0 + 0.1 * torch.randn(dim, generator=g, device="cuda")

    def step(self, ids, u, **settings):
        n = ids.shape[0]
        x = bqm.q4_dequantize(self.table, ids, scale=math.sqrt(self.dim), dtype=BF16)
        a, x = bqm.rms_norm_q8_1(x, self.gain)
        y = bqm.mm_tq1_0(self.w, a, self.dim, self.dim, n)
        a, x = bqm.rms_norm_q8_1(x, self.gain, add=y)
        logits = bqm.mm_q4(self.head, a)
        return (x, logits, *bqm.sample(logits, u, **settings))


def plain_values(m):
    b = m.codes.cpu().view(m.N, -1, 16)
    v = torch.cat((b & 15, b >> 4), -1).double()
    v = torch.where(v > 7, v - 16, v).view(m.N, m.K // m.group, m.group)
    if m.zeros is not None:
        v = v - m.zeros.cpu().double().unsqueeze(-1)
    return (v * m.scales.cpu().double().unsqueeze(-1)).flatten(1)


def dequantized(a, dim):
    b = a.cpu().view(a.shape[0], dim // 32, 36)
    q = b[..., :32].contiguous().view(torch.int8).double()
    return (q * b[..., 32:34].contiguous().view(torch.float16).double()).flatten(1)


@pytest.mark.parametrize("n", [1, 3, 20, 70])
def test_step_against_64_bits(n):
    e = Ends()
    g = torch.Generator(device="cuda").manual_seed(n)
    ids = torch.randint(0, e.vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
    u = torch.rand(n, generator=g, device="cuda")
    k, p = torch.full((n,), 40, device="cuda", dtype=torch.int32), torch.full((n,), 0.9, device="cuda")
    x, logits, tokens, logprobs = e.step(ids, u, top_k=k, top_p=p)
    # the same steps one by one, each from the one before it as the library left it
    rows = (plain_values(e.table)[ids.cpu().long()] * float(torch.tensor(math.sqrt(e.dim), dtype=F32))).float().to(BF16)
    got = bqm.q4_dequantize(e.table, ids, scale=math.sqrt(e.dim), dtype=BF16)
    assert torch.equal(got.cpu(), rows)
    a, _ = bqm.rms_norm_q8_1(got, e.gain)
    norm = rows.double() / (rows.double().square().mean(-1, keepdim=True) + 1e-6).sqrt() * e.gain.cpu().double()
    # a value is off by half a step of its block's scale, that by its rounding to 16 bits
    scale = norm.view(n, -1, 32).abs().amax(-1, keepdim=True) / 127
    room = (0.5 * (1 + 1e-4) * scale + 2.0 ** -11 * norm.view(n, -1, 32).abs() + 2.0 ** -25 * 127).reshape(n, -1)
    assert bool(((dequantized(a, e.dim) - norm).abs() <= room).all())
    y = bqm.mm_tq1_0(e.w, a, e.dim, e.dim, n)
    assert torch.equal(x, (got.float() + y).to(BF16))
    a, _ = bqm.rms_norm_q8_1(got, e.gain, add=y)
    w, c = plain_values(e.head), dequantized(a, e.dim)
    assert bool(((logits.cpu().double() - c @ w.t()).abs() <= 1e-5 * (c.abs() @ w.abs().t())).all())
    for i in range(n):
        v, order = torch.sort(logits[i].cpu().double(), descending=True, stable=True)
        s = torch.softmax(v[:40], 0)
        keep = int((torch.cumsum(s, 0) < float(p[i])).sum()) + 1
        s = s[:keep] / s[:keep].sum()
        at = min(int((torch.cumsum(s, 0) <= float(u[i])).sum()), keep - 1)
        assert int(tokens[i]) == int(order[at])
        assert abs(float(logprobs[i]) - math.log(float(s[at]))) <= 1e-6


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("n", [1, 5, 40, 130])
def test_step_captured(n):
    # a step as a graph, replayed with other tokens and numbers, eager steps between the replays; and a
    # second graph of the same sizes, replayed in turn with the first
    e = Ends(vocab=5003)
    ids = torch.zeros(n, device="cuda", dtype=torch.int32)
    u = torch.zeros(n, device="cuda")
    settings = dict(temperature=torch.full((n,), 0.8, device="cuda"), top_p=torch.full((n,), 0.95, device="cuda"),
                    min_p=torch.full((n,), 0.01, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        e.step(ids, u, **settings)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = e.step(ids, u, **settings)
        graphs.append((g, out))
    for turn in range(6):
        ids.copy_(torch.randint(0, e.vocab, (n,), device="cuda", dtype=torch.int32))
        u.copy_(torch.rand(n, device="cuda"))
        g, out = graphs[turn % 2]
        g.replay()
        want = e.step(ids, u, **settings)
        torch.cuda.synchronize()
        assert same(out, want), turn


def test_calls_on_other_streams():
    # the same calls on two streams at once, each with its own workspaces and outputs
    e = Ends(vocab=20011)
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = []
    for i in range(2):
        n = (40, 3)[i]
        a = bqm.q8_1_quantize(torch.randn(n, e.dim, device="cuda"))
        sets.append((a, torch.rand(n, device="cuda"), torch.randn(n, e.dim, device="cuda")))
    want = []
    for a, u, x in sets:
        logits = bqm.mm_q4(e.head, a)
        want.append((logits, *bqm.sample(logits, u), *bqm.rms_norm_q8_1(x, e.gain)))
    torch.cuda.synchronize()
    got = [[], []]
    for turn in range(8):
        for i, (a, u, x) in enumerate(sets):
            logits = bqm.mm_q4(e.head, a, stream=streams[i])
            with torch.cuda.stream(streams[i]):
                got[i].append((logits, *bqm.sample(logits, u, stream=streams[i]),
                               *bqm.rms_norm_q8_1(x, e.gain, stream=streams[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert same(g, want[i])


def test_a_stream_of_another_device_is_refused():
    e = Ends()

    class Other:
        stream_id, device_index, device_type, cuda_stream = 0, 1, 1, 0
    with pytest.raises(ValueError):
        bqm.mm_q4(e.head, bqm.q8_1_quantize(torch.randn(1, e.dim, device="cuda")), stream=Other())


def test_given_workspaces_and_outputs():
    # workspaces with anything in them, and no byte behind what is asked for touched
    e = Ends(vocab=80021)
    for n in (1, 40, 200):
        a = bqm.q8_1_quantize(torch.randn(n, e.dim, device="cuda"))
        u = torch.rand(n, device="cuda")
        logits = bqm.mm_q4(e.head, a)
        tokens = bqm.sample(logits, u)
        for fill in (0x00, 0xff):
            need = bqm.mm_q4_workspace_bytes(e.head, n)
            ws = torch.full((need + 512,), fill, device="cuda", dtype=torch.uint8)
            out = torch.full((n + 2, e.vocab), float("nan"), device="cuda")
            bqm.mm_q4(e.head, a, out=out[1:-1], workspace=ws[:max(need, 1)])
            assert torch.equal(out[1:-1], logits) and bool(torch.isnan(out[0]).all()) and bool(torch.isnan(out[-1]).all())
            assert bool((ws[need:] == fill).all())
            need = bqm.sample_workspace_bytes(n, e.vocab)
            ws = torch.full((need + 512,), fill, device="cuda", dtype=torch.uint8)
            t, lp = bqm.sample(logits, u, workspace=ws[:max(need, 1)])
            assert torch.equal(t, tokens[0]) and torch.equal(lp, tokens[1]) and bool((ws[need:] == fill).all())
    need = bqm.sample_workspace_bytes(1, 80021)
    assert need > 0
    with pytest.raises(ValueError):
        bqm.sample(torch.randn(1, 80021, device="cuda"), u[:1], workspace=torch.empty(need - 1, device="cuda", dtype=torch.uint8))


def test_results_do_not_depend_on_the_turn():
    # sums of shared rows and parts are the same each time
    e = Ends(vocab=30011, dim=1024)
    a = bqm.q8_1_quantize(torch.randn(48, 1024, device="cuda"))
    first = bqm.mm_q4(e.head, a)
    u = torch.rand(48, device="cuda")
    p = torch.full((48,), 0.97, device="cuda")
    tokens = bqm.sample(first, u, top_p=p)
    for _ in range(10):
        logits = bqm.mm_q4(e.head, a)
        assert torch.equal(logits, first)
        assert same(bqm.sample(logits, u, top_p=p), tokens)


def test_rows_behind_the_last_stay():
    e = Ends()
    out = torch.full((6, e.dim), 7.0, device="cuda")
    bqm.q4_dequantize(e.table, torch.tensor([3, 5], device="cuda", dtype=torch.int32), dtype=F32, out=out[2:4])
    assert bool((out[:2] == 7).all()) and bool((out[4:] == 7).all()) and not bool((out[2:4] == 7).all())
    x = torch.randn(3, e.dim, device="cuda")
    buf = torch.full((5, e.dim), 7.0, device="cuda")
    q = torch.full((5, e.dim // 32 * 36), 7, device="cuda", dtype=torch.uint8)
    bqm.rms_norm(x, out=buf[1:4])
    bqm.rms_norm_q8_1(x, out=q[1:4])
    for t in (buf, q):
        assert bool((t[0] == 7).all()) and bool((t[4] == 7).all())
