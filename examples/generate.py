"""Text in token ids, served: several samples of one prompt, a token at a time.

    x = table[id] * sqrt(dim)                q4_dequantize (the table in 4 bits)
    x = the decoder's layers                 decoder_layer.py
    logits = W . quantize(norm(x) * gain)    rms_norm_q8_1, mm_q4 (the output matrix in 4 bits)
    id = one of the likely tokens            sample

    python examples/generate.py [--prompt 200 --samples 4 --tokens 32 --temperature 0.8 --top-p 0.9]
"""
import argparse
import math
import time

import torch

from decoder_layer import Decoder, bqm


class Generator:
    """A decoder between a table and an output matrix, both kept in 4 bits."""

    def __init__(self, vocab=32000, seed=0, **decoder):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.decoder = Decoder(seed=seed, **decoder)
        self.dim, self.seqs = self.decoder.dim, self.decoder.pages.lens.shape[0]
        self.table = bqm.q4_quantize(torch.randn(vocab, self.dim, generator=gen, device="cuda") / self.dim ** 0.5)
        self.head = bqm.q4_quantize(torch.randn(vocab, self.dim, generator=gen, device="cuda") * 4.0 / self.dim ** 0.5)
        self.gain = torch.ones(self.dim, device="cuda")
        self.random = gen

    def logits(self, ids, new):
        """After new[s] tokens of each sequence s, ids int32 in order: the logits of each
        sequence's last one."""
        x = bqm.q4_dequantize(self.table, ids, scale=math.sqrt(self.dim), dtype=torch.float32)
        last = torch.tensor(new).cumsum(0)[torch.tensor(new) > 0] - 1
        x = self.decoder.step(x, new)[last.cuda()]
        a, _ = bqm.rms_norm_q8_1(x, self.gain)
        return bqm.mm_q4(self.head, a)

    def draw(self, logits, **settings):
        u = torch.rand(logits.shape[0], generator=self.random, device="cuda")
        return bqm.sample(logits, u, **settings)

    def generate(self, prompt, samples, tokens, temperature=0.8, top_k=0, top_p=1.0, min_p=0.0):
        """(ids int32 [samples, tokens], the sum of each one's logprobs): the prompt is
        sequence 0 and its samples are forks of it."""
        full = lambda v, t=torch.float32: torch.full((samples,), v, dtype=t, device="cuda")  # noqa: E731
        settings = dict(temperature=full(temperature), top_k=full(top_k, torch.int32), top_p=full(top_p), min_p=full(min_p))
        logits = self.logits(prompt, [prompt.shape[0]] + [0] * (self.seqs - 1)).expand(samples, -1).contiguous()
        if samples > 1:
            self.decoder.fork([0] * (samples - 1), list(range(1, samples)))
        ids, logprobs = [], 0.0
        for i in range(tokens):
            new, lp = self.draw(logits, **settings)
            ids.append(new)
            logprobs = logprobs + lp
            if i + 1 < tokens:
                logits = self.logits(new, [1] * samples + [0] * (self.seqs - samples))
        return torch.stack(ids, 1), logprobs


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=200, help="tokens of the prompt")
    ap.add_argument("--samples", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=32, help="of each sample")
    ap.add_argument("--temperature", type=float, default=0.8)
    ap.add_argument("--top-k", type=int, default=0)
    ap.add_argument("--top-p", type=float, default=0.9)
    ap.add_argument("--min-p", type=float, default=0.0)
    a = ap.parse_args()
    g = Generator(layers=a.layers)
    if not 1 <= a.samples <= g.seqs or a.prompt < 1 or a.tokens < 1 or a.prompt + a.tokens > 64 * 16:
        ap.error("the example's table holds %d sequences of 1024 tokens" % g.seqs)
    prompt = torch.randint(0, g.table.N, (a.prompt,), generator=g.random, device="cuda", dtype=torch.int32)
    t = time.perf_counter()
    ids, logprobs = g.generate(prompt, a.samples, a.tokens, a.temperature, a.top_k, a.top_p, a.min_p)
    torch.cuda.synchronize()
    print("%d samples of %d tokens behind a prompt of %d: %.1f ms" % (*ids.shape, a.prompt, (time.perf_counter() - t) * 1e3))
    for row, lp in zip(ids.cpu().tolist(), logprobs.cpu().tolist()):
        print("logprob %8.2f:" % lp, *row[:12], "..." if len(row) > 12 else "")


if __name__ == "__main__":
    main()
