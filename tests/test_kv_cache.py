"""The cache's bookkeeping on the CPU: no GPU, no library."""
import pytest
import torch

from orthogonal_reparameterized_02_amd.attention import KVCache


def rows(n, start=0.0):
    return torch.arange(n * 8, dtype=torch.float32).view(n, 1, 8) + start


def test_cache_in_host_memory():
    cache = KVCache(2, 4, 1, 8, dtype=torch.float32, device="cpu")
    cache.fill(0, rows(3), rows(3, 100))
    assert cache.longest() == 3
    cache.append(rows(2, 500), rows(2, 600))
    assert cache.length.tolist() == [4, 1] and torch.equal(cache.k[0, 3], rows(2, 500)[0]) and torch.equal(cache.v[1, 0], rows(2, 600)[1])
    with pytest.raises(ValueError, match="full"):
        cache.append(rows(2), rows(2))
    cache.fill(0, rows(0), rows(0))
    cache.append(rows(2), rows(2))
    assert cache.length.tolist() == [1, 2] and cache.longest() == 2
    with pytest.raises(ValueError, match="fit"):
        cache.fill(1, rows(5), rows(5))


def test_caches_without_sequences_or_rows():
    none = KVCache(0, 4, 1, 8, dtype=torch.float32, device="cpu")
    none.append(rows(0), rows(0))
    assert none.longest() == 0
    flat = KVCache(1, 0, 1, 8, dtype=torch.float32, device="cpu")
    with pytest.raises(ValueError, match="full"):
        flat.append(rows(1), rows(1))
