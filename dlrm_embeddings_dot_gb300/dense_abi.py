"""Constants and C signatures of ``include/dlrm_dense.h``.  Needs ctypes alone, so that the library
loads, and its host-only calls run, without torch."""

from __future__ import annotations

import ctypes

DLRM_ACT_NONE = 0
DLRM_ACT_RELU = 1
DLRM_ACT_GELU = 2
DLRM_ACT_SILU = 3
DLRM_MOE_MAX_TOKENS = 64
DLRM_MOE_MAX_EXPERTS = 256
DLRM_MOE_MAX_TOP_K = 8

_P, _I, _L, _D, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double, ctypes.c_size_t

_SIGNATURES = {
    "dlrm_dropout_fwd": (_I, [_P, _L, _P, _L, _I, _I, _I, _D, _P, _P, _L, _P]),
    "dlrm_dropout_bwd": (_I, [_P, _L, _I, _I, _I, _D, _P, _P, _L, _P]),
    "dlrm_linear_fwd": (_I, [_P, _L, _P, _L, _P, _P, _L, _I, _I, _I, _I, _I, _D, _P, _P, _L, _P, _L, _P, _Z, _P, _P]),
    "dlrm_linear_fwd_workspace_size": (_Z, [_P, _L, _P, _L, _I, _I, _I, _I]),
    "dlrm_linear_bwd": (_I, [_P, _L, _P, _L, _P, _L, _P, _L, _I, _I, _I, _I, _I, _D, _P, _P, _L, _P, _L, _P, _P, _Z,
                             _P, _P]),
    "dlrm_linear_bwd_workspace_size": (_Z, [_P, _L, _P, _L, _P, _L, _I, _I, _I, _I, _I, _D]),
    "dlrm_moe_fwd": (_I, [_P, _L, _P, _P, _P, _P, _L, _I, _I, _I, _I, _I, _I, _I, _I, _P, _L, _P, _P, _P, _Z, _P, _P]),
    "dlrm_moe_fwd_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I]),
}


def declare(lib) -> None:
    """Sets the C signatures of the entry points on a loaded library."""
    for name, (res, args) in _SIGNATURES.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
