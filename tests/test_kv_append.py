"""One token more for every sequence of a cache in 4 bits: a batch of another
size is refused before anything is written or counted.  CPU only: the kernel's
calls are recorded, not run."""
import pytest
import torch

from orthogonal_reparameterized_02_amd import attention as A


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kw", [{}, dict(window=60, sinks=2)])
@pytest.mark.parametrize("n", [0, 1, 2, 4])
def test_a_batch_of_another_size(n, kw, captured, monkeypatch):
    calls = []
    monkeypatch.setattr(A.P, "poetx_kv4_write", lambda k, v, *a, **b: calls.append(tuple(k.shape)))
    cache = A.KVCache4(3, 64, 1, 8, dtype=torch.float32, device="cpu", **kw)
    monkeypatch.setattr(cache, "_captured", lambda: captured)
    good, bad = torch.zeros(3, 1, 8), torch.zeros(n, 1, 8)
    for k, v in ((bad, bad), (bad, good), (good, bad)):
        with pytest.raises(ValueError, match="3 sequences"):
            cache.append(k, v)
    assert cache.length.tolist() == [0, 0, 0] and not calls and cache._filled == [0, 0, 0] and cache._appended == 0
    cache.append(good, good)
    assert cache.length.tolist() == [1, 1, 1] and calls == [(3, 1, 8)]
