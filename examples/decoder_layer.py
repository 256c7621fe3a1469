"""Decoder layers with ternary weights, served: a prompt in chunks, a decode step
for several sequences at once, samples that branch off, sequences that end and a
cache that is moved together.

Each layer is the library's quantized products around its attention side:

    q, k, v = W_qkv . quantize(norm(x))      mm_tq1_0 (or mmvq_tq1_0)
    q, cache <- rope(q), rope(k), v          rope_kv_append
    a = attention(q, cache)                  paged_attention, fp32 out
    x = x + W_out . quantize(a)              mmvq_tq1_0_add
    x = x + W_down . quantize(silu(W_gate . n) * (W_up . n)),  n = quantize(norm(x))

    python examples/decoder_layer.py [--layers 4 --tokens 600 --steps 16]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_mat_amd as bqm  # noqa: E402


class Matrix:
    """A ternary matrix [N, K] packed as TQ1_0."""

    def __init__(self, N, K, gen):
        self.N, self.K = N, K
        trits = torch.randint(-1, 2, (N, K), generator=gen, device="cuda", dtype=torch.int8)
        scale = torch.full((N, K // 256), 1.2 / K ** 0.5, device="cuda", dtype=torch.float16)
        self.w = bqm.tq1_pack(trits, scale)

    def __call__(self, a, T, add=None):
        if add is not None and T <= bqm.MMVQ_MAX_COLS:
            return bqm.mmvq_tq1_0_add(self.w, a, add, self.N, self.K, T)
        y = bqm.mm_tq1_0(self.w, a, self.N, self.K, T)
        return y if add is None else y.add_(add)


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Decoder:
    """Layers, their cache and the sequences in it."""

    def __init__(self, layers=2, dim=1024, heads=8, kv_heads=2, hidden=2816, pages=256, page_size=16,
                 max_seqs=8, max_pages=64, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.dim, self.heads, self.kv_heads, self.head = dim, heads, kv_heads, dim // heads
        self.hidden, self.page_size = hidden, page_size
        self.layers = [dict(qkv=Matrix((heads + 2 * kv_heads) * self.head, dim, gen),
                            out=Matrix(dim, dim, gen), gate=Matrix(hidden, dim, gen),
                            up=Matrix(hidden, dim, gen), down=Matrix(dim, hidden, gen))
                       for _ in range(layers)]
        shape = (layers, pages, page_size, kv_heads, self.head)
        self.cache = bqm.KvCache(torch.empty(shape, dtype=dtype, device="cuda"),
                                 torch.empty(shape, dtype=dtype, device="cuda"))
        self.caches = [self.cache.layer(i) for i in range(layers)]
        self.angles = bqm.rope_table(bqm.rope_inv_freq(self.head), max_pages * page_size)
        self.pages = bqm.KvPages(torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device="cuda"),
                                 torch.zeros(max_seqs, dtype=torch.int32, device="cuda"),
                                 torch.zeros(pages, dtype=torch.int32, device="cuda"))

    def _take(self, pages, short_of):
        """The new state, if every sequence got its pages: one that did not keeps its old
        length, and new tokens would be stored over its last ones. (A server counts the
        free pages on the host; here the answer is waited for.)"""
        self.short_of = short_of
        if int(short_of):
            raise RuntimeError("no free pages for %d sequences" % int(short_of))
        self.pages = pages

    def step(self, x, new):
        """x fp32 [tokens, dim]: new[s] tokens of each sequence s, in order. Their
        states after all layers, attended over everything before them."""
        n_new = torch.tensor(new, dtype=torch.int32)
        starts = torch.cat((torch.zeros(1, dtype=torch.int32), n_new.cumsum(0, dtype=torch.int32)))
        self._take(*bqm.kv_extend(self.pages, n_new.cuda(), self.page_size))
        batch = bqm.KvBatch(self.pages.table, self.pages.lens, starts.cuda(), max_q=max(new))
        T, H, G = x.shape[0], self.heads, self.kv_heads
        for layer, cache in zip(self.layers, self.caches):
            row = layer["qkv"](bqm.q8_1_quantize(norm(x)), T).view(T, H + 2 * G, self.head)
            q = bqm.rope_kv_append(row[:, :H], row[:, H:H + G], row[:, H + G:], cache, batch, self.angles)
            a = bqm.paged_attention(q, cache, batch, out_dtype=torch.float32)
            x = layer["out"](bqm.q8_1_quantize(a.view(T, self.dim)), T, add=x)
            n = bqm.q8_1_quantize(norm(x))
            if T <= bqm.GLU_MAX_COLS:
                h = bqm.mmvq_tq1_0_glu(layer["gate"].w, layer["up"].w, n, self.hidden, self.dim, T)
            else:
                h = torch.nn.functional.silu(layer["gate"](n, T)) * layer["up"](n, T)
            x = layer["down"](bqm.q8_1_quantize(h), T, add=x)
        return x

    def fork(self, parents, children):
        """Sequences children (empty ones) go on from where parents are."""
        p, c = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (parents, children))
        pages, moves, short_of = bqm.kv_fork(self.pages, p, c, self.page_size)
        self._take(pages, short_of)
        bqm.kv_copy_pages(self.cache, moves)

    def end(self, seqs):
        self.pages = bqm.kv_free(self.pages, torch.tensor(seqs, dtype=torch.int32, device="cuda"))

    def compact(self):
        self.pages, moves, _ = bqm.kv_compact(self.pages, self.page_size)
        bqm.kv_copy_pages(self.cache, moves)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=600, help="of the prompt")
    ap.add_argument("--chunk", type=int, default=256)
    ap.add_argument("--steps", type=int, default=16, help="decode steps")
    a = ap.parse_args()
    if a.tokens < 1 or a.tokens + a.steps + 1 > 64 * 16:
        ap.error("the example's table holds 1024 tokens a sequence")
    d = Decoder(layers=a.layers)
    x = torch.randn(a.tokens, d.dim, device="cuda")
    seqs = d.pages.lens.shape[0]
    t = time.perf_counter()
    for at in range(0, a.tokens, a.chunk):  # sequence 0, a chunk at a time
        n = min(a.chunk, a.tokens - at)
        last = d.step(x[at:at + n], [n] + [0] * (seqs - 1))[-1:]
    torch.cuda.synchronize()
    print("prompt of %d tokens in chunks of %d: %.1f ms" % (a.tokens, a.chunk, (time.perf_counter() - t) * 1e3))
    d.fork([0, 0, 0], [1, 2, 3])  # three more samples of the same prompt
    y = last.repeat(4, 1)
    t = time.perf_counter()
    for _ in range(a.steps):
        y = d.step(norm(y) + 0.1 * torch.randn_like(y), [1] * 4 + [0] * (seqs - 4))
    torch.cuda.synchronize()
    print("%d steps of 4 sequences: %.2f ms a step" % (a.steps, (time.perf_counter() - t) * 1e3 / max(1, a.steps)))
    d.end([0, 2])
    used = int((d.pages.refs > 0).sum())
    d.compact()
    print("2 of 4 ended: %d pages in use, the last of them %d" % (used, int(d.pages.refs.nonzero().max())))
    y = d.step(norm(y[1::2]), [0, 1, 0, 1] + [0] * (seqs - 4))
    print("one more step of the others: finite %s, pages short %d" % (bool(torch.isfinite(y).all()), int(d.short_of)))


if __name__ == "__main__":
    main()
