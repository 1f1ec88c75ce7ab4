"""Binding of ``include/dlrm_dense.h``: the dense layer and its gradient, dropout and the
mixture-of-experts layer for a few tokens.

As in the package, every function has the name of the C entry point it calls and fills the
output tensors it is given.  Sizes and row distances come from the tensors: matrices are 2-D
with unit column stride (rows may be further apart than their width), of one dtype (fp32,
fp16 or bf16); biases and their gradients are fp32 vectors; ``rng`` is an int64 tensor of two
elements (seed, offset) on the device.
"""

from __future__ import annotations

import ctypes

import torch

import dlrm_embeddings_dot_gb300 as _dl

DLRM_ACT_NONE = 0
DLRM_ACT_RELU = 1
DLRM_ACT_GELU = 2
DLRM_ACT_SILU = 3
DLRM_MOE_MAX_TOKENS = 64
DLRM_MOE_MAX_EXPERTS = 256
DLRM_MOE_MAX_TOP_K = 8

_CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_P, _I, _L, _D, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double, ctypes.c_size_t
_fn = {}

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


def _call(name, *args):
    f = _fn.get(name)
    if f is None:
        f = _fn[name] = getattr(_dl.load(), name)
    rc = f(*args)
    if rc:
        raise _dl.DlrmError(name, rc, _dl.dlrm_last_error())


def _size(name, *args) -> int:
    return int(getattr(_dl.load(), name)(*args))


def _current_stream():
    """Handle of torch's current stream.  Asked for without the Stream object around it, which
    costs 3 us on the host where the whole call of a small layer is to cost about 6."""
    if torch.cuda.is_initialized():
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return torch.cuda.current_stream().cuda_stream


def _stream(stream):
    return _current_stream() if stream is None else _dl._stream(stream)


def _code(dt) -> int:
    c = _CODE.get(dt)
    if c is None:
        raise TypeError(f"unsupported dtype {dt}")
    return c


def _mat(name, t, shape, dt):
    """(address, row distance) of a matrix argument of this shape and dtype; (None, 0) for None."""
    if t is None:
        return None, 0
    if t.dtype is not dt:
        raise TypeError(f"{name} is {t.dtype}, not {dt}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    ld, unit = t.stride()
    if unit != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), ld


def _dense(name, t, shape, dt):
    """Address of a contiguous argument of this shape; None for None."""
    if t is None:
        return None
    if t.dtype is not dt:
        raise TypeError(f"{name} is {t.dtype}, not {dt}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous of shape {shape}")
    return t.data_ptr()


def _rng(rng):
    return None if rng is None else _dense("rng", rng, (2,), torch.int64)


def _ws(workspace):
    return (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)


def dlrm_dropout_fwd(x, residual, y, p, rng, stream=None):
    """y = residual + drop(x) (residual may be None); see ``include/dlrm_dense.h``."""
    M, N = x.shape
    dt = x.dtype
    _call("dlrm_dropout_fwd", *_mat("x", x, (M, N), dt), *_mat("residual", residual, (M, N), dt), _code(x.dtype), M, N, p,
          _rng(rng), *_mat("y", y, (M, N), dt), _stream(stream))


def dlrm_dropout_bwd(grad_y, grad_x, p, rng, stream=None):
    """grad_x = drop(grad_y) with the mask of the forward that had the same p and rng."""
    M, N = grad_y.shape
    dt = grad_y.dtype
    _call("dlrm_dropout_bwd", *_mat("grad_y", grad_y, (M, N), dt), _code(grad_y.dtype), M, N, p, _rng(rng),
          *_mat("grad_x", grad_x, (M, N), dt), _stream(stream))


def dlrm_linear_fwd_workspace_size(x, w) -> int:
    (M, K), N = x.shape, w.shape[0]
    return _size("dlrm_linear_fwd_workspace_size", *_mat("x", x, (M, K), x.dtype), *_mat("w", w, (N, K), x.dtype),
                 _code(x.dtype), M, N, K)


def dlrm_linear_fwd(x, w, bias, residual, y, pre=None, act=DLRM_ACT_NONE, p=0.0, rng=None, workspace=None, status=None,
                    stream=None):
    """y = residual + drop(act(x w^T + bias)), the pre-activation to ``pre`` where given; bias and
    residual may be None.  See ``include/dlrm_dense.h``."""
    M, K = x.shape
    N = w.shape[0]
    dt = x.dtype
    _call("dlrm_linear_fwd", *_mat("x", x, (M, K), dt), *_mat("w", w, (N, K), dt), _dense("bias", bias, (N,), torch.float32),
          *_mat("residual", residual, (M, N), dt), _code(x.dtype), M, N, K, act, p, _rng(rng), *_mat("y", y, (M, N), dt),
          *_mat("pre", pre, (M, N), dt), *_ws(workspace), _dl._ptr(status), _stream(stream))


def dlrm_linear_bwd_workspace_size(grad_y, x, w, act=DLRM_ACT_NONE, p=0.0) -> int:
    (M, K), N, dt = x.shape, w.shape[0], x.dtype
    return _size("dlrm_linear_bwd_workspace_size", *_mat("grad_y", grad_y, (M, N), dt), *_mat("x", x, (M, K), dt),
                 *_mat("w", w, (N, K), dt), _code(x.dtype), M, N, K, act, p)


def dlrm_linear_bwd(grad_y, x, w, pre, grad_x, grad_w, grad_bias, act=DLRM_ACT_NONE, p=0.0, rng=None, workspace=None,
                    status=None, stream=None):
    """Gradients of ``dlrm_linear_fwd``; each of grad_x, grad_w, grad_bias may be None.  See
    ``include/dlrm_dense.h``."""
    M, K = x.shape
    N = w.shape[0]
    dt = x.dtype
    _call("dlrm_linear_bwd", *_mat("grad_y", grad_y, (M, N), dt), *_mat("x", x, (M, K), dt), *_mat("w", w, (N, K), dt),
          *_mat("pre", pre, (M, N), dt), _code(x.dtype), M, N, K, act, p, _rng(rng), *_mat("grad_x", grad_x, (M, K), dt),
          *_mat("grad_w", grad_w, (N, K), dt), _dense("grad_bias", grad_bias, (N,), torch.float32), *_ws(workspace),
          _dl._ptr(status), _stream(stream))


def _moe_sizes(x, w_router, w1, w2):
    T, H = x.shape
    return T, H, w2.shape[2], w_router.shape[0]


def dlrm_moe_fwd_workspace_size(x, w_router, w1, w2, top_k) -> int:
    T, H, I, E = _moe_sizes(x, w_router, w1, w2)
    return _size("dlrm_moe_fwd_workspace_size", _code(x.dtype), T, H, I, E, top_k)


def dlrm_moe_fwd(x, w_router, w1, w2, residual, y, ids, probs, act=DLRM_ACT_SILU, gated=True, workspace=None,
                 status=None, stream=None):
    """Mixture-of-experts layer for a few tokens: y = residual + sum of probs * expert(x) over the
    top-k experts (k from ids [T][k]); residual may be None.  See ``include/dlrm_dense.h``."""
    T, H, I, E = _moe_sizes(x, w_router, w1, w2)
    dt, k = x.dtype, ids.shape[1]
    _call("dlrm_moe_fwd", *_mat("x", x, (T, H), dt), _dense("w_router", w_router, (E, H), dt),
          _dense("w1", w1, (E, 2 * I if gated else I, H), dt), _dense("w2", w2, (E, H, I), dt),
          *_mat("residual", residual, (T, H), dt), _code(x.dtype), T, H, I, E, k, act, bool(gated),
          *_mat("y", y, (T, H), dt), _dense("ids", ids, (T, k), torch.int32),
          _dense("probs", probs, (T, k), torch.float32), *_ws(workspace), _dl._ptr(status), _stream(stream))
