"""The bookkeeping of a ring cache on the CPU: no GPU, no library."""
import pytest
import torch

from orthogonal_reparameterized_02_amd.attention import AttentionPlan, KVCache


def ring(rows=8, sinks=3, window=5, B=2):
    return KVCache(B, rows, 1, 8, dtype=torch.float32, device="cpu", window=window, sinks=sinks)


def tokens(n, start=0):
    return torch.arange(start, start + n, dtype=torch.float32)[:, None, None].expand(n, 1, 8).contiguous()


def first_and_newest(n, rows=8, sinks=3):
    return list(range(n)) if n <= rows else [*range(sinks), *range(n - (rows - sinks), n)]


@pytest.mark.parametrize("n", [0, 1, 2, 3, 4, 7, 8, 9, 13, 14, 40])
def test_ring_filled_by_a_prompt(n):
    cache = ring()
    cache.fill(1, tokens(n), tokens(n, 100))
    k, v = cache.held(1)
    assert k[:, 0, 0].tolist() == first_and_newest(n) and v[:, 0, 0].tolist() == [100 + i for i in first_and_newest(n)]
    assert cache.length.tolist() == [0, n] and cache.tokens(1) == n and cache.longest() == n


@pytest.mark.parametrize("parts", [[1] * 30, [2, 1, 9, 4], [8, 8, 8], [3, 5, 1], [20, 3], [2, 30], [0, 4, 0, 11]])
def test_ring_extended_and_appended(parts):
    cache, at = ring(), 0
    for n in parts:
        cache.extend(0, tokens(n, at), tokens(n, at + 100))
        at += n
        k, v = cache.held(0)
        assert k[:, 0, 0].tolist() == first_and_newest(at) and v[:, 0, 0].tolist() == [100 + i for i in first_and_newest(at)]
    for i in range(13):  # every sequence's next token, never full
        cache.append(torch.stack([tokens(1, at + i)[0], tokens(1, i)[0]]), torch.zeros(2, 1, 8))
        assert cache.held(0)[0][:, 0, 0].tolist() == first_and_newest(at + i + 1)
        assert cache.held(1)[0][:, 0, 0].tolist() == first_and_newest(i + 1)
    assert cache.tokens(0) == at + 13 and cache.tokens(1) == 13


def test_ring_without_sinks_and_slots_filled_again():
    cache = ring(rows=4, sinks=0, window=4)
    cache.fill(0, tokens(10), tokens(10))
    assert cache.held(0)[0][:, 0, 0].tolist() == [6, 7, 8, 9]
    cache.fill(0, tokens(2, 50), tokens(2, 50))
    assert cache.held(0)[0][:, 0, 0].tolist() == [50, 51] and cache.longest() == 2


def test_plain_cache_extended():
    cache = KVCache(1, 6, 1, 8, dtype=torch.float32, device="cpu")
    cache.fill(0, tokens(2), tokens(2))
    cache.extend(0, tokens(3, 2), tokens(3, 2))
    assert cache.held(0)[0][:, 0, 0].tolist() == [0, 1, 2, 3, 4] and cache.length.tolist() == [5]
    with pytest.raises(ValueError, match="fit"):
        cache.extend(0, tokens(2), tokens(2))
    assert cache.length.tolist() == [5]


@pytest.mark.parametrize("kw", [dict(window=-1), dict(sinks=-1, window=4), dict(sinks=2), dict(window=5, sinks=4)])
def test_ring_refusals(kw):
    with pytest.raises(ValueError):
        KVCache(1, 8, 1, 8, dtype=torch.float32, device="cpu", **kw)


def test_plan_refusals():
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="prefixes"):
        AttentionPlan(cu, 4, prefix=cu[:1], window=2)
    with pytest.raises(ValueError, match="sinks"):
        AttentionPlan(cu, 4, sinks=2)


def test_counts_are_refused_while_a_graph_is_captured(monkeypatch):
    """A replay would take the count of now: nothing that reads one on the host
    is captured, and the cache stays as it was."""
    cache = ring()
    cache.fill(0, tokens(5), tokens(5))
    monkeypatch.setattr(cache, "_captured", lambda: True)
    for call in (lambda: cache.tokens(0), lambda: cache.held(0), lambda: cache.extend(0, tokens(1), tokens(1))):
        with pytest.raises(RuntimeError, match="captured"):
            call()
    assert cache.length.tolist() == [5, 0]
