"""How many sequences and heads a decoding call takes: as many as its launch
can have workgroups, 32 query heads of a key head each."""
import ctypes as C
import os

import pytest
import torch

from orthogonal_reparameterized_02_amd import _lib
from orthogonal_reparameterized_02_amd import poetx as P
from test_abi_block import FAKE, OUT, decode_shape

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libpoetx.so not built")


def shape(B, Hq, Hkv, rows=2):
    return decode_shape(B=B, Hq=Hq, Hkv=Hkv, D=8, act=1, rows=rows, ldq=8 * Hq, ldo=8 * Hq, ldk=8 * Hkv, ldv=8 * Hkv,
                        bsk=8 * Hkv * rows, bsv=8 * Hkv * rows)


@pytest.mark.parametrize("B,Hq,Hkv", [(65535, 512, 32), (65535, 1024, 128), (65535, 256, 256), (16384, 1023, 1023)])
def test_large_calls_are_taken(B, Hq, Hkv):
    assert _lib.lib().poetx_attn_decode_workspace_bytes(C.byref(shape(B, Hq, Hkv))) >= B * Hq * 8 * 4


@pytest.mark.parametrize("B,Hq,Hkv", [(65535, 512, 512), (16384, 1024, 1024), (65535, 1022, 511)])
def test_a_grid_of_two_to_the_32_threads_is_refused(B, Hq, Hkv):
    L, sh = _lib.lib(), shape(B, Hq, Hkv)
    assert L.poetx_attn_decode_workspace_bytes(C.byref(sh)) == 0
    assert L.poetx_attn_decode(C.byref(sh), FAKE, FAKE, FAKE, None, FAKE, None, OUT, FAKE, 1 << 60, None) == 1
    assert "2^24" in L.poetx_last_error().decode()


@pytest.mark.gpu
def test_many_sequences_of_many_heads():
    """2^25 rows of queries, 2^20 workgroups: every one's answer, and what is
    behind the last row left as it was."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B, Hq, Hkv, D, rows = 65535, 512, 16, 8, 2
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    q, k, v = randn(B, Hq, D), randn(B, rows, Hkv, D), randn(B, rows, Hkv, D)
    length = (torch.arange(B, device="cuda") % 3).int()
    out = torch.full((B + 1, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    sh = P.decode_shape(q, k, v)
    ws = torch.empty(P.poetx_attn_decode_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    P.poetx_attn_decode(sh, q, k, v, length, out[:B], ws)
    worst = 0.0
    for b in range(0, B, 8192):
        e = min(b + 8192, B)
        qs = q[b:e].float().view(e - b, Hkv, Hq // Hkv, D)
        s = torch.stack([(qs * k[b:e, j].float()[:, :, None]).sum(-1) for j in range(rows)], -1) / D ** 0.5
        s[torch.arange(rows, device="cuda").expand_as(s) >= length[b:e, None, None, None]] = float("-inf")
        p = torch.softmax(s, -1).nan_to_num(0.0)  # none seen: 0
        want = sum(p[..., j:j + 1] * v[b:e, j].float()[:, :, None] for j in range(rows)).view(e - b, Hq, D)
        got = out[b:e].float()
        # one rounding of the result, 2^-8 of it at most; p in two bf16 parts and
        # float32 sums of a few terms below 8 lie under 2^-12
        assert ((got - want).abs() <= want.abs() * 2.0 ** -8 + 2.0 ** -12).all()
        worst = max(worst, (got - want).abs().max().item())
    assert worst > 0 and (out[B] == 7).all() and not out[0].any()
