"""Which sequence a cache's calls mean: counted from the end below 0, refused
where there is none, alike for both forms.  CPU only: the 4-bit form's kernel
calls are recorded, not run."""
import pytest
import torch

from orthogonal_reparameterized_02_amd import attention as A

FORMS = [A.KVCache, A.KVCache4]


def rows(n, start=0.0):
    return torch.arange(n * 8, dtype=torch.float32).view(n, 1, 8) + start


@pytest.fixture
def calls(monkeypatch):
    """The sequences that kernel calls name."""
    seen = []
    monkeypatch.setattr(A.P, "poetx_kv4_write", lambda k, v, seq, pos, *cache, **kw: seen.append(seq.tolist()))
    monkeypatch.setattr(A.P, "poetx_kv4_read", lambda seq, pos, *a, **kw: seen.append(seq.tolist()))
    return seen


def cache_of(form, **kw):
    return form(3, 64, 1, 8, dtype=torch.float32, device="cpu", **kw)


@pytest.mark.parametrize("kw", [{}, dict(window=60, sinks=2)])
@pytest.mark.parametrize("form", FORMS)
def test_sequences_from_the_end(form, kw, calls):
    cache = cache_of(form, **kw)
    cache.fill(-1, rows(4), rows(4))
    cache.extend(-1, rows(3), rows(3))
    cache.fill(-3, rows(2), rows(2))
    assert cache.length.tolist() == [2, 0, 7] and cache.tokens(-1) == cache.tokens(2) == 7 and cache.longest() == 7
    k, _ = cache.held(-1)
    assert k.shape == (7, 1, 8)
    if form is A.KVCache4:
        assert calls == [[2] * 4, [2] * 3, [0] * 2, [2] * 7]
    else:
        assert torch.equal(k, torch.cat([rows(4), rows(3)])) and torch.equal(cache.k[0, :2], rows(2))


@pytest.mark.parametrize("b", [3, -4, 2 ** 32])
@pytest.mark.parametrize("form", FORMS)
def test_sequences_that_are_not_there(form, b, calls):
    cache = cache_of(form)
    cache.fill(0, rows(4), rows(4))
    for call in (lambda: cache.fill(b, rows(2), rows(2)), lambda: cache.fill(b, rows(0), rows(0)),
                 lambda: cache.extend(b, rows(2), rows(2)), lambda: cache.tokens(b), lambda: cache.held(b)):
        with pytest.raises(IndexError):
            call()
    assert cache.length.tolist() == [4, 0, 0] and cache.longest() == 4 and len(calls) == (form is A.KVCache4)
