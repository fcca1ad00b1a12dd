"""The last sequence of a cache named from its end, on the GPU."""
import pytest
import torch

from orthogonal_reparameterized_02_amd import attention as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    A.P.lib()


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("form", [A.KVCache, A.KVCache4])
def test_a_prompt_of_the_last_sequence(form, window):
    """The same values, and the same answers, as by its place from the front."""
    g = torch.Generator(device="cuda").manual_seed(window)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)
    k, v, q = randn(50, 2, 64), randn(50, 2, 64), randn(3, 4, 64)
    got = []
    for b in (2, -1):
        cache = form(3, 64, 2, 64, window=window)
        for t in vars(cache).values():  # what is not written is NaN
            if torch.is_tensor(t) and t.dim() == 4:
                t.fill_(255) if t.dtype == torch.uint8 else t.fill_(float("nan"))
        cache.fill(b, k[:30], v[:30])
        cache.extend(b, k[30:], v[30:])
        got.append((*cache.held(b), A.attention_decode(q, cache), cache.length))
    assert got[1][3].tolist() == [0, 0, 50]
    assert torch.isfinite(got[1][0]).all() and torch.isfinite(got[1][2]).all() and got[1][2][2].any()
    for x, y in zip(*got):
        assert torch.equal(x, y)
