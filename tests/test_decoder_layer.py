"""The example's decoder: what the library's products and its attention side give
together must not depend on how the tokens were fed or where their pages lie."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import decoder_layer
    finally:
        sys.path.pop(0)
    return decoder_layer


def _decoder(example, **kw):
    return example.Decoder(**{**dict(layers=2, dim=512, heads=4, kv_heads=2, hidden=768, pages=64, max_seqs=4,
                                     max_pages=16), **kw})


def test_chunks_give_what_the_whole_prompt_gives(example):
    x = torch.randn(150, 512, generator=torch.Generator().manual_seed(1)).cuda()
    whole = _decoder(example).step(x, [0, 150, 0, 0])
    d = _decoder(example)
    parts = torch.cat([d.step(x[a:b], [0, b - a, 0, 0]) for a, b in ((0, 70), (70, 71), (71, 100), (100, 150))])
    # the same tokens through other kernels: a weight rounds to 16 bits against
    # another base (2^-8 of it at most), and a value near a step of the 8-bit
    # activations (1/127 of its block's largest) may fall to the other side; both
    # average out over the rows of the products
    rel = float((parts - whole).norm() / whole.norm())
    assert rel < 0.02, rel


def test_forks_and_compaction_keep_what_a_sequence_sees(example):
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(100, 512, generator=gen).cuda()
    y = torch.randn(1, 512, generator=gen).cuda()
    d = _decoder(example)
    d.step(x[:30], [30, 0, 0, 0])
    d.step(x, [0, 100, 0, 0])
    d.fork([1, 1], [2, 3])
    out = d.step(y.repeat(3, 1), [0, 1, 1, 1])
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
    d.end([0, 1])
    d.compact()
    used = int((d.pages.refs > 0).sum())
    assert int(d.pages.refs.nonzero().max()) == used - 1
    # the same next token for the two that are left, and for one that was never
    # forked or moved
    moved = d.step(y.repeat(2, 1), [0, 0, 1, 1])
    e = _decoder(example)
    e.step(x, [0, 100, 0, 0])
    e.step(y, [0, 1, 0, 0])
    plain = e.step(y, [0, 1, 0, 0])
    assert torch.equal(moved[0], moved[1])
    assert float((moved[0] - plain[0]).norm() / plain[0].norm()) < 0.02
    assert int(d.short_of) == 0


def test_example_runs(example, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["decoder_layer.py", "--layers", "1", "--tokens", "70", "--steps", "2"])
    example.main()
    assert "finite True, pages short 0" in capsys.readouterr().out
