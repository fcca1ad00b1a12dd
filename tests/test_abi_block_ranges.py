"""The attention entry points refuse sizes that their kernels' integers and
launches cannot hold.  CPU only: nothing here reaches a device."""
import ctypes as C
import os

import pytest

from orthogonal_reparameterized_02_amd import _lib
from test_abi_block import FAKE, OUT, attn_shape, decode_shape

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libpoetx.so not built")

ROWS = 2 ** 31 - 2 ** 16
ONE = dict(Hq=1, Hkv=1, D=8, ldq=8, ldk=8, ldv=8, ldo=8, lddo=8, lddq=8, lddk=8, lddv=8)


@pytest.mark.parametrize("kw,word", [
    (dict(Tq=ROWS + 1, Tk=1), "Tq="), (dict(Tq=1, Tk=ROWS + 1), "Tk="), (dict(Tq=2 ** 31 - 1, Tk=2 ** 31 - 1), "Tk="),
    (dict(Tq=2 ** 31 - 200, Tk=0), "above"),
    # more threads than one launch can have
    (dict(Tq=2 ** 26, Tk=1, Hq=32, ldq=256, ldo=256, lddo=256, lddq=256), "Hq=32"),
    (dict(Tq=1, Tk=2 ** 24 - 100, Hq=128, Hkv=128, **{n: 1024 for n in ("ldq", "ldk", "ldv", "ldo", "lddo", "lddq", "lddk", "lddv")}), "Hkv=128"),
])
def test_attention_refuses_sizes_past_its_integers(kw, word):
    L = _lib.lib()
    sh = attn_shape(**{**ONE, **kw})
    assert L.poetx_attn_plan_bytes(C.byref(sh)) == 0
    assert L.poetx_attn_workspace_bytes(C.byref(sh), 1) == 0
    for st in (L.poetx_attn_plan(C.byref(sh), FAKE, FAKE, None, FAKE, 1 << 60, None),
               L.poetx_attn_fwd(C.byref(sh), FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, 1 << 60, None),
               L.poetx_attn_bwd(C.byref(sh), *[FAKE] * 6, None, *[FAKE] * 5, 1 << 60, None)):
        assert st == 1 and word in L.poetx_last_error().decode()


def test_attention_takes_the_largest_sizes():
    L = _lib.lib()
    sh = attn_shape(**{**ONE, "Tq": ROWS, "Tk": ROWS})
    assert L.poetx_attn_plan_bytes(C.byref(sh)) >= 20 * ROWS
    assert L.poetx_attn_workspace_bytes(C.byref(sh), 1) >= 8 * ROWS
    sh = attn_shape(**{**ONE, "Tq": 2 ** 26 - 128, "Tk": 1, "Hq": 32, **{n: 256 for n in ("ldq", "ldo", "lddo", "lddq")}})
    assert L.poetx_attn_workspace_bytes(C.byref(sh), 1) >= 8 * 32 * (2 ** 26 - 128)


def test_decode_refuses_caches_past_its_integers():
    L = _lib.lib()
    one = dict(B=1, Hq=1, Hkv=1, D=8, ldq=8, ldo=8, ldk=8, ldv=8, bsk=0, bsv=0)
    for rows in (ROWS + 1, 2 ** 31 - 1):
        sh = decode_shape(**one, rows=rows)
        assert L.poetx_attn_decode_workspace_bytes(C.byref(sh)) == 0
        assert L.poetx_attn_decode(C.byref(sh), FAKE, FAKE, FAKE, None, FAKE, None, OUT, FAKE, 1 << 40, None) == 1
        assert "rows=" in L.poetx_last_error().decode()
    assert L.poetx_attn_decode_workspace_bytes(C.byref(decode_shape(**one, rows=ROWS))) > 0
