"""Binding of ``include/dlrm_dense.h``: the dense layer and its gradient, dropout and the
mixture-of-experts layer for a few tokens.

As in the package, every function has the name of the C entry point it calls and fills the
output tensors it is given.  Sizes and row distances come from the tensors: matrices are 2-D
with unit column stride (rows may be further apart than their width), of one dtype (fp32,
fp16 or bf16); biases and their gradients are fp32 vectors; ``rng`` is an int64 tensor of two
elements (seed, offset).  Every tensor is on the current device, ``rng``, ``workspace`` and
``status`` too (ValueError otherwise).
"""

from __future__ import annotations

import ctypes

import torch

import dlrm_embeddings_dot_gb300 as _dl

from .dense_abi import (DLRM_ACT_GELU, DLRM_ACT_NONE, DLRM_ACT_RELU, DLRM_ACT_SILU, DLRM_MOE_MAX_EXPERTS,  # noqa: F401
                        DLRM_MOE_MAX_TOKENS, DLRM_MOE_MAX_TOP_K, declare)

_TYPES = (torch.float32, torch.float16, torch.bfloat16, torch.int32, torch.int64)
_marshal = None


def _load():
    """The checking extension (csrc/marshal.c), bound to the library's entry points."""
    global _marshal
    if _marshal is None:
        lib = _dl.load()
        try:
            from . import _marshal as m
        except ImportError as e:
            raise RuntimeError("the _marshal extension is missing: build the library first "
                               "(python -c 'import __graft_entry__ as g; g.build()'), with a C compiler and Python's "
                               "headers") from e
        names = ("dlrm_dropout_fwd", "dlrm_dropout_bwd", "dlrm_linear_fwd", "dlrm_linear_bwd", "dlrm_moe_fwd")
        m.bind(_TYPES, torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device,
               torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream")
               else lambda d: torch.cuda.current_stream(d).cuda_stream,
               tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names))
        _marshal = m
    return _marshal


def _fail(name, rc):
    raise _dl.DlrmError(name, rc, _dl.dlrm_last_error())


def _handle(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def _size(name, *args) -> int:
    return int(getattr(_dl.load(), name)(*args))


def _code(dt) -> int:
    if dt not in _TYPES[:3]:
        raise TypeError(f"unsupported dtype {dt}")
    return _TYPES.index(dt)


def _at(t):
    """(address, row distance) of a matrix whose shape has been read."""
    return t.data_ptr(), t.stride(0)


def dlrm_dropout_fwd(x, residual, y, p, rng, stream=None):
    """y = residual + drop(x) (residual may be None); see ``include/dlrm_dense.h``."""
    rc = (_marshal or _load()).dropout_fwd(x, residual, y, p, rng, _handle(stream))
    if rc:
        _fail("dlrm_dropout_fwd", rc)


def dlrm_dropout_bwd(grad_y, grad_x, p, rng, stream=None):
    """grad_x = drop(grad_y) with the mask of the forward that had the same p and rng."""
    rc = (_marshal or _load()).dropout_bwd(grad_y, grad_x, p, rng, _handle(stream))
    if rc:
        _fail("dlrm_dropout_bwd", rc)


def dlrm_linear_fwd_workspace_size(x, w) -> int:
    (M, K), N = x.shape, w.shape[0]
    return _size("dlrm_linear_fwd_workspace_size", *_at(x), *_at(w), _code(x.dtype), M, N, K)


def dlrm_linear_fwd(x, w, bias, residual, y, pre=None, act=DLRM_ACT_NONE, p=0.0, rng=None, workspace=None, status=None,
                    stream=None):
    """y = residual + drop(act(x w^T + bias)), the pre-activation to ``pre`` where given; bias and
    residual may be None.  See ``include/dlrm_dense.h``."""
    rc = (_marshal or _load()).linear_fwd(x, w, bias, residual, y, pre, act, p, rng, workspace, status, _handle(stream))
    if rc:
        _fail("dlrm_linear_fwd", rc)


def dlrm_linear_bwd_workspace_size(grad_y, x, w, act=DLRM_ACT_NONE, p=0.0) -> int:
    (M, K), N = x.shape, w.shape[0]
    return _size("dlrm_linear_bwd_workspace_size", *_at(grad_y), *_at(x), *_at(w), _code(x.dtype), M, N, K, act, p)


def dlrm_linear_bwd(grad_y, x, w, pre, grad_x, grad_w, grad_bias, act=DLRM_ACT_NONE, p=0.0, rng=None, workspace=None,
                    status=None, stream=None):
    """Gradients of ``dlrm_linear_fwd``; each of grad_x, grad_w, grad_bias may be None.  See
    ``include/dlrm_dense.h``."""
    rc = (_marshal or _load()).linear_bwd(grad_y, x, w, pre, grad_x, grad_w, grad_bias, act, p, rng, workspace, status,
                                          _handle(stream))
    if rc:
        _fail("dlrm_linear_bwd", rc)


def dlrm_moe_fwd_workspace_size(x, w_router, w1, w2, top_k) -> int:
    (T, H), I, E = x.shape, w2.shape[2], w_router.shape[0]
    return _size("dlrm_moe_fwd_workspace_size", _code(x.dtype), T, H, I, E, top_k)


def dlrm_moe_fwd(x, w_router, w1, w2, residual, y, ids, probs, act=DLRM_ACT_SILU, gated=True, workspace=None,
                 status=None, stream=None):
    """Mixture-of-experts layer for a few tokens: y = residual + sum of probs * expert(x) over the
    top-k experts (k from ids [T][k]); residual may be None.  See ``include/dlrm_dense.h``."""
    rc = (_marshal or _load()).moe_fwd(x, w_router, w1, w2, residual, y, ids, probs, act, gated, workspace, status,
                                       _handle(stream))
    if rc:
        _fail("dlrm_moe_fwd", rc)
