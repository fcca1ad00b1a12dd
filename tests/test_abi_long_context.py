"""The long-context entry points reject bad arguments on the host before
anything reaches a device.  CPU only: every call here fails validation or has
nothing to do, so no kernel is launched."""
import ctypes as C
import os

import pytest
import torch

from orthogonal_reparameterized_02_amd import _lib
from orthogonal_reparameterized_02_amd import poetx as P

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libpoetx.so not built")

FAKE = C.c_void_p(0x10000)      # aligned, never dereferenced
OUT = C.c_void_p(0x20000)
MISALIGNED = C.c_void_p(0x10002)


def _err():
    return _lib.lib().poetx_last_error().decode()


# ---- norms of queries and keys ------------------------------------------------------
def norm_shape(**kw):
    a = dict(T=4, Hq=4, Hk=2, D=64, rot=64, P=16, act=1, interleaved=0, eps=1e-6, ldq=256, ldk=128, ldqo=256,
             ldko=128, lddq=256, lddk=128)
    a.update(kw)
    return _lib.QkNormShape(**a)


FWD = ("q", "k", "wq", "wk", "pos", "table", "qo", "ko")
BWD = ("dqo", "dko", "q", "k", "wq", "wk", "pos", "table", "dq", "dk", "dwq", "dwk")


def fwd(sh, **kw):
    a = {n: OUT if n in ("qo", "ko") else FAKE for n in FWD} | kw
    return _lib.lib().poetx_qk_norm_rope_fwd(C.byref(sh) if sh else None, *[a[n] for n in FWD], None)


def bwd(sh, ws=FAKE, n=1 << 40, **kw):
    a = {n: OUT if n in ("dq", "dk") else FAKE for n in BWD} | kw
    return _lib.lib().poetx_qk_norm_rope_bwd(C.byref(sh) if sh else None, *[a[n] for n in BWD], ws, n, None)


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), "T="), (dict(Hq=0), "Hq="), (dict(Hk=-1), "Hk="), (dict(Hq=2000), "Hq="), (dict(P=0), "P="),
    (dict(D=60), "D="), (dict(D=520), "D="), (dict(rot=-2), "rot="), (dict(rot=33), "rot="), (dict(rot=66), "rot="),
    (dict(act=2), "dtype"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"),
    (dict(ldq=255), "ldq"), (dict(ldk=132), "ldk"), (dict(ldqo=128), "ldqo"), (dict(ldko=1 << 25), "ldko")])
def test_norm_shape_errors(kw, word):
    sh = norm_shape(**kw)
    assert fwd(sh) == 1 and word in _err()
    assert bwd(sh) == 1 and word in _err()
    assert _lib.lib().poetx_qk_norm_rope_workspace_bytes(C.byref(sh)) == 0


def test_norm_pointer_errors_and_nothing_to_do():
    assert fwd(None) == 1 and bwd(None) == 1
    for call, names in ((fwd, FWD), (bwd, BWD)):
        for n in names:
            assert call(norm_shape(), **{n: MISALIGNED}) == 1 and f"'{n}'" in _err()
            if not n.startswith(("w", "dw")):
                assert call(norm_shape(), **{n: None}) == 1 and f"'{n}'" in _err()
    for kw in (dict(lddq=8), dict(lddk=132)):
        assert bwd(norm_shape(**kw)) == 1 and next(iter(kw)) in _err()
    assert fwd(norm_shape(ldqo=264), qo=FAKE) == 1 and "in place" in _err()
    assert bwd(norm_shape(lddq=264), dq=FAKE) == 1 and "in place" in _err()
    need = _lib.lib().poetx_qk_norm_rope_workspace_bytes(C.byref(norm_shape()))
    assert need > 0 and bwd(norm_shape(), n=need - 1) == 3 and bwd(norm_shape(), ws=None) == 1
    assert fwd(norm_shape(T=0), q=None) == 0
    assert bwd(norm_shape(T=0), q=None, ws=None, dwq=None, dwk=None) == 0


def test_norm_binding_refusals():
    q = torch.zeros(4, 2, 16)
    t, pos = torch.zeros(8, 8, 2), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        P.poetx_qk_norm_rope_fwd(q, None, None, None, pos, t, q, None)
    with pytest.raises(ValueError, match="table"):
        P.poetx_qk_norm_rope_fwd(q, None, None, None, pos, t[0], q, None)
    with pytest.raises(ValueError, match="unsupported activation"):
        P.qk_norm_shape(q.double(), None, None)
