"""Constants and C signatures of ``include/dlrm_block.h``.  Needs ctypes alone, so that the library
loads, and its host-only calls run, without torch."""

from __future__ import annotations

import ctypes

DLRM_NORM_RMS = 0
DLRM_NORM_LAYER = 1
DLRM_GATE_NONE = 0
DLRM_GATE_SIGMOID = 1
DLRM_GATE_SILU = 2
DLRM_BLOCK_MAX_WIDTH = 8192
DLRM_ROUTE_MAX_EXPERTS = 256
DLRM_ROUTE_MAX_TOP_K = 8

# in the order in which the checking extension takes their addresses
ENTRY_POINTS = ("dlrm_block_norm_fwd", "dlrm_block_norm_bwd", "dlrm_route_fwd", "dlrm_route_bwd", "dlrm_expert_sort",
                "dlrm_dispatch_fwd", "dlrm_dispatch_bwd", "dlrm_combine_fwd", "dlrm_combine_bwd", "dlrm_pack8",
                "dlrm_unpack8", "dlrm_linear_bwd8")
SIZES = ("dlrm_block_norm_bwd_workspace_size", "dlrm_expert_sort_workspace_size", "dlrm_linear_bwd8_workspace_size")

_P, _I, _L, _D, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double, ctypes.c_size_t
_M = [_P, _L]    # a matrix: address and row distance

_SIGNATURES = {
    "dlrm_block_norm_fwd": (_I, _M * 2 + [_I] + _M + [_P] * 5 + [_I] * 5 + [_D] + _M * 2 + [_P] * 2),
    "dlrm_block_norm_bwd": (_I, _M * 4 + [_I] + _M + [_P] * 5 + [_I] * 5 + _M * 3 + [_P] * 6 + [_Z, _P]),
    "dlrm_block_norm_bwd_workspace_size": (_Z, [_I, _I]),
    "dlrm_route_fwd": (_I, _M + [_I] * 4 + [_P] * 3),
    "dlrm_route_bwd": (_I, [_P] * 3 + [_I] * 4 + _M + [_P]),
    "dlrm_expert_sort": (_I, [_P] + [_I] * 3 + [_P] * 4 + [_Z, _P, _P]),
    "dlrm_expert_sort_workspace_size": (_Z, [_I] * 3),
    "dlrm_dispatch_fwd": (_I, _M + [_P] + [_I] * 5 + _M + [_P] * 2),
    "dlrm_dispatch_bwd": (_I, _M + [_P] + [_I] * 5 + _M + [_P] * 2),
    "dlrm_combine_fwd": (_I, _M + [_P] * 2 + _M + [_I] * 5 + _M + [_P] * 2),
    "dlrm_combine_bwd": (_I, _M * 2 + [_P] * 2 + [_I] * 5 + _M + [_P] * 3),
    "dlrm_pack8": (_I, _M + [_I] * 3 + _M + [_P] * 2),
    "dlrm_unpack8": (_I, _M + [_P] + [_I] * 3 + _M + [_P]),
    "dlrm_linear_bwd8": (_I, _M * 2 + [_P] + _M * 2 + [_P] + [_I] * 5 + [_D, _P] + _M * 2 + [_P] * 2 + [_Z, _P, _P]),
    "dlrm_linear_bwd8_workspace_size": (_Z, _M * 2 + [_I] * 5 + [_D]),
}


def declare(lib) -> None:
    """Sets the C signatures of the entry points on a loaded library."""
    for name, (res, args) in _SIGNATURES.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
