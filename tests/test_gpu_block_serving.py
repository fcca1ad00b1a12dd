"""The attention block's module and cache in use: slots filled again, captured
decoding steps, positions past the table, recomputation, second derivatives.
Tolerances as in test_gpu_block.py."""
import pytest
import torch

from orthogonal_reparameterized_02_amd import attention as A
from test_gpu_attention_block import randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# ---- the cache ---------------------------------------------------------------------------
def test_a_cache_slot_is_filled_again():
    """A full sequence makes way for a short one; the others' room is their
    own, and an emptied slot takes none of it."""
    cache, kv = A.KVCache(2, 6, 1, 64), lambda n, s=0: randn(n, 1, 64, seed=s)
    cache.fill(0, kv(6), kv(6, 1))
    cache.fill(1, kv(2), kv(2, 1))
    with pytest.raises(ValueError, match="full"):
        cache.append(kv(2), kv(2))
    cache.fill(0, kv(3, 2), kv(3, 3))
    for i in range(3):
        cache.append(kv(2, 4 + i), kv(2, 14 + i))
    assert cache.length.tolist() == [6, 5]
    assert torch.equal(cache.k[0, 3:, 0], torch.cat([kv(2, 4 + i)[:1, 0] for i in range(3)]))
    assert torch.equal(cache.v[1, 2:5, 0], torch.cat([kv(2, 14 + i)[1:, 0] for i in range(3)]))
    with pytest.raises(ValueError, match="full"):
        cache.append(kv(2), kv(2))
    cache.fill(0, kv(0), kv(0))
    cache.append(kv(2), kv(2))
    assert cache.length.tolist() == [1, 6]
