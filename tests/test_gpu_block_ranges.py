"""GPU parity of the attention-block operators at the ends of their ranges,
against the float64 oracle; tolerances as in test_gpu_block.py."""
import pytest
import torch

from orthogonal_reparameterized_02_amd import poetx as P
from test_gpu_block import DT, check, reference, run, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    P.lib()


# ---- distances -----------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("cap", [0.0, 6.0])
def test_bias_past_row_2_24(dt, cap):
    """A short document behind more rows than float32 can count."""
    first = 2 ** 24 + 37
    st = setup(dict(q=[50], k=[61], Hq=1, Hkv=1, D=8, cap=cap, bias=True), dt)
    ref, _ = reference(st)
    for n in ("k", "v"):
        st[n] = torch.cat([torch.zeros(first, 1, 8, dtype=DT[dt], device="cuda"), st[n]])
    st["cu_k"] = st["cu_k"] + first
    out = run(st)
    for n in ("dk", "dv"):
        assert not out[n][:first].any()
        out[n] = out[n][first:]
    check(out, ref, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_bias_of_query_rows_past_2_24(dt):
    """The same with the query rows there too."""
    first = 2 ** 24 + 5
    st = setup(dict(q=[70], k=[70], Hq=1, Hkv=1, D=8, bias=True), dt)
    ref, _ = reference(st)
    for n in ("q", "k", "v", "dout"):
        st[n] = torch.cat([torch.zeros(first, 1, 8, dtype=DT[dt], device="cuda"), st[n]])
    st["cu_q"], st["cu_k"] = st["cu_q"] + first, st["cu_k"] + first
    out = run(st)
    for n in ("o", "dq", "dk", "dv"):
        assert not out[n][:first].any()
        out[n] = out[n][first:]
    assert torch.isneginf(out["lse"][:, :first]).all()
    out["lse"] = out["lse"][:, first:]
    check(out, ref, dt)
