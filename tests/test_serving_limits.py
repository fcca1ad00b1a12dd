"""The rotary table ends for a ring as for any cache, and counts idle slots."""
import pytest
import torch

from orthogonal_reparameterized_02_amd import attention as A

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("four", [False, True])
def test_a_ring_at_the_end_of_the_table(four):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    block = A.POETXAttention(256, 4, 2, 32, k=3, positions=100, qk_norm=True, window=24, sinks=2).eval()
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda n: torch.randn(n, 256, generator=g, device="cuda").bfloat16()
    cache = block.cache(2, 100, four)
    assert cache.ring
    block.prefill(randn(60), cache, 0)
    block.prefill(randn(39), cache, 0, follow=True)
    assert torch.isfinite(block.decode(randn(2), cache)).all() and cache.length.tolist() == [100, 1]
    with pytest.raises(ValueError, match="positions"):  # sequence 0, used or idle, has no position left
        block.decode(randn(2), cache)
    with pytest.raises(ValueError, match="positions"):
        block.prefill(randn(1), cache, 0, follow=True)
    assert cache.length.tolist() == [100, 1]
    none = torch.empty(0, 2, block.D, dtype=torch.bfloat16, device="cuda")
    cache.fill(0, none, none)
    assert torch.isfinite(block.decode(randn(2), cache)).all() and cache.length.tolist() == [1, 2]
