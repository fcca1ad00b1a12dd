"""Norms of queries and keys at the ends of what float32 sums of squares hold:
128 equal elements sum to 2^128 from 2^60.5 on.

Heads that fit are normed to float32 (here to 2^-20: some twenty roundings of 2^-24)
and rounded once (bf16 2^-8); a head that does not is written as zeros, with
gradients of zero, and takes nothing from its neighbours."""
import pytest
import torch

from orthogonal_reparameterized_02_amd import attention as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    A.P.lib()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_large_and_small_heads(dt):
    tol = 2.0 ** -20 if dt == torch.float32 else 2.0 ** -8 + 2.0 ** -20
    sign = torch.where(torch.arange(128, device="cuda") % 3 == 0, -1.0, 1.0)
    powers = [60, 61, 64, 100, 120, 0, -30, -60, -62]
    heads = torch.stack([sign * 2.0 ** p for p in powers])[None].to(dt)
    q = heads.clone().requires_grad_()
    w = torch.ones(128, device="cuda", requires_grad=True)
    y = A.qk_norm_rope(q, None, w, None, None, None, eps=0.0)
    big = torch.tensor([p > 60 for p in powers], device="cuda")
    assert (y[0, big] == 0).all()
    assert ((y[0, ~big].float() - sign).abs() <= tol).all()
    g = torch.zeros_like(y)
    g[..., 0] = 1.0
    y.backward(g)
    assert (q.grad[0, big] == 0).all()
    # r (g - n mean(g n)): n = -1 in element 0, its sign elsewhere, mean(g n) = -1 / 128
    for i, p in enumerate(powers):
        if p <= 60:
            want = 2.0 ** -p * ((torch.arange(128, device="cuda") == 0).float() + sign / 128)
            assert ((q.grad[0, i].float() - want).abs() <= tol * 2.0 ** -p).all(), p
    assert abs(w.grad[0].item() + (~big).sum().item()) <= 2.0 ** -18 and not w.grad[1:].any()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_gradients_whose_products_pass_the_range(dt):
    """The sum of dy w x is 2^6 * 2^125 * 128: NaN in that head alone."""
    q = torch.full((1, 3, 128), 1.0, device="cuda", dtype=dt)
    q[0, 1] = 2.0 ** 125
    q.requires_grad_()
    w = torch.ones(128, device="cuda", requires_grad=True)
    y = A.qk_norm_rope(q, None, w, None, None, None)
    y.backward(torch.full_like(y, 64.0))
    assert (y[0, 1] == 0).all() and torch.isnan(q.grad[0, 1]).all()
    assert torch.isfinite(q.grad[0, [0, 2]]).all() and torch.isfinite(w.grad).all()
