"""ctypes loader for libpoetx.so (built in-tree by build.py).

The library is the only compute path: if it is missing the calls raise; there
is no fallback.
"""
from __future__ import annotations

import ctypes as C
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpoetx.so")

F32, BF16 = 0, 1
I8 = 2  # weight storage only (fold, dequant)
STATUS = {0: "POETX_OK", 1: "POETX_ERR_ARG", 2: "POETX_ERR_UNSUPPORTED",
          3: "POETX_ERR_WORKSPACE", 4: "POETX_ERR_DEVICE"}

# every symbol include/poetx.h declares, with its ctypes signature
_p, _i, _sz = C.c_void_p, C.c_int32, C.c_size_t
_i64, _u64, _d = C.c_int64, C.c_uint64, C.c_double
SIGNATURES = {
    "poetx_abi_version": (_i, []),
    "poetx_status_str": (C.c_char_p, [_i]),
    "poetx_last_error": (C.c_char_p, []),
    "poetx_cnp_fwd": (_i, [_i, _i, _i, _p, _p, _p, _i, _p, _sz, _p]),
    "poetx_cnp_fwd_noalloc": (_i, [_i, _i, _i, _p, _p, _p, _i, _p]),
    "poetx_cnp_bwd": (_i, [_i, _i, _i, _p, _p, _p, _i, _i, _p, _sz, _p]),
    "poetx_cnp_bwd_after_fwd": (_i, [_i, _i, _i, _p, _p, _p, _i, _i, _p, _sz, _p]),
    "poetx_cnp_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "poetx_fold_perm": (_i, [_i, _i, _i, _p, _p, _p, _p, _p, _p, _p, _p]),
    "poetx_layer_fwd": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "poetx_layer_bwd": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "poetx_workspace_bytes": (_sz, [_p, _i]),
    "poetx_saved_bytes": (_sz, [_p]),
    "poetx_layer_fwd_xmem": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "poetx_layer_bwd_xmem": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _sz,
                                  _p]),
    "poetx_saved_bytes_xmem": (_sz, [_p]),
    "poetx_merge": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "poetx_layer_fwd_q": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _i, _p]),
    "poetx_layer_bwd_q": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _sz,
                               _i, _p]),
    "poetx_fold_scale": (_i, [_i, _p, _p, _p, _p]),
    "poetx_dequant": (_i, [_i, _i, _p, _p, _i, _p, _p]),
    "poetx_set_stage_events": (_i, [_p, _i]),
    "poetx_set_fused_gather": (_i, [_i]),
    "poetx_rope": (_i, [_p, _p, _p, _p, _p, _p, _p, _p]),
    "poetx_qk_norm_rope_workspace_bytes": (_sz, [_p]),
    "poetx_qk_norm_rope_fwd": (_i, [_p] * 10),
    "poetx_qk_norm_rope_bwd": (_i, [_p] * 14 + [_sz, _p]),
    "poetx_dropout_fwd": (_i, [_i64, _i, _p, _p, _p, _d, _u64, _u64, _p, _p]),
    "poetx_dropout_bwd": (_i, [_i64, _i, _p, _p, _d, _u64, _u64, _p, _p]),
    "poetx_attn_plan_bytes": (_sz, [_p]),
    "poetx_attn_workspace_bytes": (_sz, [_p, _i]),
    "poetx_attn_plan": (_i, [_p, _p, _p, _p, _p, _sz, _p]),
    "poetx_attn_fwd": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "poetx_attn_bwd": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "poetx_attn_window_plan_bytes": (_sz, [_p, _p]),
    "poetx_attn_window_workspace_bytes": (_sz, [_p, _p, _i]),
    "poetx_attn_window_plan": (_i, [_p, _p, _p, _p, _p, _sz, _p]),
    "poetx_attn_window_fwd": (_i, [_p] * 10 + [_sz, _p]),
    "poetx_attn_window_bwd": (_i, [_p] * 14 + [_sz, _p]),
    "poetx_attn_decode_workspace_bytes": (_sz, [_p]),
    "poetx_attn_decode": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "poetx_attn_window_decode_workspace_bytes": (_sz, [_p, _p]),
    "poetx_attn_window_decode": (_i, [_p, _p, _i] + [_p] * 7 + [_sz, _p]),
    "poetx_kv4_write": (_i, [_p] * 10),
    "poetx_kv4_read": (_i, [_p] * 10),
    "poetx_attn_kv4_decode_workspace_bytes": (_sz, [_p, _p]),
    "poetx_attn_kv4_decode": (_i, [_p, _p, _i] + [_p] * 10 + [_sz, _p]),
}


NOALLOC_SCRATCH_BYTES = 32 << 20  # POETX_NOALLOC_SCRATCH_BYTES
ABI_VERSION = 2                   # POETX_ABI_VERSION


class Shape(C.Structure):
    _fields_ = [("m", C.c_int32), ("n", C.c_int32), ("b", C.c_int32), ("k", C.c_int32),
                ("T", C.c_int32), ("act", C.c_int32)]


def _struct(name: str, ints: str, floats: str, longs: str):
    fields = ([(f, C.c_int32) for f in ints.split()] + [(f, C.c_float) for f in floats.split()]
              + [(f, C.c_int64) for f in longs.split()])
    return type(name, (C.Structure,), {"_fields_": fields})


RopeShape = _struct("RopeShape", "T Hq Hk D rot P act interleaved inverse", "",
                    "ldq ldk ldqo ldko")
QkNormShape = _struct("QkNormShape", "T Hq Hk D rot P act interleaved", "eps",
                      "ldq ldk ldqo ldko lddq lddk")
AttnShape = _struct("AttnShape", "Tq Tk ndoc Hq Hkv D act causal", "scale cap",
                    "ldq ldk ldv ldo lddo lddq lddk lddv")
Kv4Shape = _struct("Kv4Shape", "T B rows Hkv D act sinks ring", "", "ldk ldv")
Window = _struct("Window", "window sinks", "", "")
DecodeShape = _struct("DecodeShape", "B Hq Hkv D act rows", "scale cap",
                      "ldq ldo ldk ldv bsk bsv")


class PoetxError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} -> {STATUS.get(status, status)}: {msg}")
        self.status = status


_lib = None


def lib() -> C.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run "
                               "`python -m orthogonal_reparameterized_02_amd.build`")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        if L.poetx_abi_version() != ABI_VERSION:
            raise RuntimeError("libpoetx.so ABI version mismatch")
        _lib = L
    return _lib


def check(fn: str, status: int) -> None:
    if status != 0:
        raise PoetxError(fn, status, lib().poetx_last_error().decode())
