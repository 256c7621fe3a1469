"""The example's decoder when its cache is full: it says so, and what is in the cache stays."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_decoder_layer import _decoder, example  # noqa: E402, F401


def _state(d):
    return [t.clone() for t in (*d.pages, d.cache.k, d.cache.v)]


def test_a_full_cache_is_an_error(example):  # noqa: F811
    x = torch.randn(40, 512, generator=torch.Generator().manual_seed(5)).cuda()
    d = _decoder(example, pages=4)
    d.cache.k.zero_(), d.cache.v.zero_()
    d.step(x, [40, 0, 0, 0])  # 3 pages
    before = _state(d)
    with pytest.raises(RuntimeError, match="1 sequences"):
        d.step(x[:30], [0, 30, 0, 0])  # two, and one is left
    with pytest.raises(RuntimeError, match="1 sequences"):
        d.fork([0, 0], [1, 2])  # a copied last page each
    assert all(torch.equal(a, b) for a, b in zip(before, _state(d)))
    d.step(x[:10], [8, 2, 0, 0])
    assert d.pages.lens.cpu().tolist() == [48, 2, 0, 0]
