"""Weights of the query and key norms are shared by all heads of a tensor: one
of another size, a weight a head among them, is refused and not read in part
(its gradient would be left unwritten behind the first D)."""
import pytest
import torch

from orthogonal_reparameterized_02_amd import attention as A
from orthogonal_reparameterized_02_amd import poetx as P

T, H, D = 4, 2, 16


def tensors(device):
    return (torch.zeros(T, H, D, device=device), torch.zeros(8, D // 2, 2, device=device),
            torch.zeros(T, dtype=torch.int32, device=device))


def check(device, shape, which):
    q, table, pos = tensors(device)
    w, good = torch.ones(*shape, device=device), torch.ones(D, device=device)
    pair = lambda bad: (bad, good) if which == "q" else (good, bad)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=device)
    with pytest.raises(ValueError, match=f"w{which} has shape"):
        P.poetx_qk_norm_rope_fwd(q, q, *pair(w), pos, table, q.clone(), q.clone())
    with pytest.raises(ValueError, match=f"w{which} has shape"):
        P.poetx_qk_norm_rope_bwd(q, q, q, q, *pair(w), pos, table, q.clone(), q.clone(), None, None, ws)
    with pytest.raises(ValueError, match=f"dw{which} has shape"):
        P.poetx_qk_norm_rope_bwd(q, q, q, q, good, good, pos, table, q.clone(), q.clone(), *pair(w), ws)
    with pytest.raises(ValueError, match=f"w{which} has shape"):
        A.qk_norm_rope(q, q, *(x.clone().requires_grad_() for x in pair(w)), pos, table)


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("shape", [(H, D), (D + 1,), (2 * D,), (D // 2,), (0,)])
def test_weights_of_another_size(shape, which):
    check("cpu", shape, which)


@pytest.mark.gpu
def test_weights_of_another_size_on_the_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    for which in "qk":
        check("cuda", (H, D), which)
    q = torch.randn(T, H, D, device="cuda")
    a = A.qk_norm_rope(q, None, torch.ones(1, D, device="cuda"), None, None, None)  # one row of D is one weight
    assert torch.equal(a, A.qk_norm_rope(q, None, torch.ones(D, device="cuda"), None, None, None)) and a.any()
