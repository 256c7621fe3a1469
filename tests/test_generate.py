"""The example that generates: its tokens are those of the steps done one by one, and greedy
samples of one prompt are alike."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMALL = dict(vocab=500, layers=1, dim=512, heads=4, kv_heads=2, hidden=768, pages=64, max_seqs=4, max_pages=16)


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import generate
    finally:
        sys.path.pop(0)
    return generate


def _prompt(n):
    return torch.randint(0, 500, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int32).cuda()


def test_greedy_samples_are_alike(example):
    ids, logprobs = example.Generator(**SMALL).generate(_prompt(37), 3, 9, temperature=0.0)
    assert ids.shape == (3, 9) and torch.equal(ids[0], ids[1]) and torch.equal(ids[0], ids[2])
    assert bool((logprobs == 0).all())
    # and each is the largest logit of the step before it
    g = example.Generator(**SMALL)
    logits = g.logits(_prompt(37), [37, 0, 0, 0])
    g.decoder.fork([0, 0], [1, 2])
    for i in range(9):
        assert int(logits[0].argmax()) == int(ids[0, i])
        if i < 8:
            logits = g.logits(ids[:, i].contiguous(), [1, 1, 1, 0])


def test_samples_stay_within_their_filters(example):
    g = example.Generator(**SMALL)
    logits = g.logits(_prompt(20), [20, 0, 0, 0]).expand(400, -1).contiguous()
    full = lambda v, t: torch.full((400,), v, dtype=t, device="cuda")  # noqa: E731
    ids, logprobs = g.draw(logits, top_k=full(7, torch.int32))
    best = set(logits[0].topk(7).indices.cpu().tolist())
    assert set(ids.cpu().tolist()) <= best and len(set(ids.cpu().tolist())) > 1
    assert bool((logprobs <= 0).all())


def test_example_runs(example, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["generate.py", "--layers", "1", "--prompt", "30", "--samples", "2", "--tokens", "5"])
    example.main()
    out = capsys.readouterr().out
    assert "2 samples of 5 tokens behind a prompt of 30" in out and out.count("logprob") == 2
