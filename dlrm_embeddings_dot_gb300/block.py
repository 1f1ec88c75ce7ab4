"""Binding of ``include/dlrm_block.h``: the norms around a block with its gate and residual scale, the
choice of experts and the order of the tokens by expert, the tokens' way to their experts and back, and
activations in 8 bits.

As in ``dense.py``, every function has the name of the C entry point it calls, fills the output tensors it
is given and checks shapes, dtypes, strides and devices first (TypeError, ValueError).  Matrices are 2-D
with unit column stride, of one dtype (fp32, fp16 or bf16); vectors, ``stats``, ``probs`` and their
gradients are fp32, ``ids``, ``slots``, ``order`` and ``offsets`` int32, all contiguous; 8-bit matrices and
their exponents are uint8.
"""

from __future__ import annotations

import dlrm_embeddings_dot_gb300 as _dl

from . import dense as _dense
from .block_abi import DLRM_GATE_NONE, DLRM_NORM_RMS
from .dense import _at, _code, _fail, _handle
from .dense import _size as _dense_size
from .dense_abi import DLRM_ACT_NONE


def _size(name, *args) -> int:
    if not hasattr(_dl.load(), name):
        raise RuntimeError(f"the library was built before {name}: build it again")
    return _dense_size(name, *args)


def dlrm_block_norm_fwd(y, gate, residual, w_post, b_post, scale, w_pre, b_pre, r, h, stats=None, norm=DLRM_NORM_RMS,
                        gate_act=DLRM_GATE_NONE, eps=1e-6, stream=None):
    """r = residual + scale * gate(g) * (norm(y) * w_post + b_post); h = norm(r) * w_pre + b_pre.  Without
    y (None) r is the residual, without h no norm of r is taken; gate is [M][N] or [M][1].  stats [M][4]
    keeps the rows' statistics for the backward.  See ``include/dlrm_block.h``."""
    rc = (_dense._marshal or _dense._load()).block_norm_fwd(y, gate, residual, w_post, b_post, scale, w_pre, b_pre, r, h, stats,
                                                            norm, gate_act, eps, _handle(stream))
    if rc:
        _fail("dlrm_block_norm_fwd", rc)


def dlrm_block_norm_bwd_workspace_size(r) -> int:
    """Bytes for rows of r's shape."""
    M, N = r.shape
    return _size("dlrm_block_norm_bwd_workspace_size", M, N)


def dlrm_block_norm_bwd(grad_r, grad_h, y, gate, r, stats, w_post, b_post, scale, w_pre, grad_y, grad_gate, grad_residual,
                        grad_w_post, grad_b_post, grad_scale, grad_w_pre, grad_b_pre, norm=DLRM_NORM_RMS,
                        gate_act=DLRM_GATE_NONE, workspace=None, stream=None):
    """Gradients of ``dlrm_block_norm_fwd``; each output may be None.  r is the forward's r (its residual
    where it had no y), None without grad_h.  See ``include/dlrm_block.h``."""
    rc = (_dense._marshal or _dense._load()).block_norm_bwd(
        grad_r, grad_h, y, gate, r, stats, w_post, b_post, scale, w_pre, grad_y, grad_gate, grad_residual, grad_w_post,
        grad_b_post, grad_scale, grad_w_pre, grad_b_pre, norm, gate_act, workspace, _handle(stream))
    if rc:
        _fail("dlrm_block_norm_bwd", rc)


def dlrm_route_fwd(logits, ids, probs, stream=None):
    """The k experts of the largest logits of each token (k from ids [T][k]) and their shares; experts
    with a logit of -infinity are closed, ids of choices that stay empty -1."""
    rc = (_dense._marshal or _dense._load()).route_fwd(logits, ids, probs, _handle(stream))
    if rc:
        _fail("dlrm_route_fwd", rc)


def dlrm_route_bwd(grad_probs, ids, probs, grad_logits, stream=None):
    """Gradient of the logits of ``dlrm_route_fwd``, 0 for experts that were not chosen."""
    rc = (_dense._marshal or _dense._load()).route_bwd(grad_probs, ids, probs, grad_logits, _handle(stream))
    if rc:
        _fail("dlrm_route_bwd", rc)


def dlrm_expert_sort_workspace_size(ids, E) -> int:
    T, k = ids.shape
    return _size("dlrm_expert_sort_workspace_size", T, k, E)


def dlrm_expert_sort(ids, E, offsets, slots, order=None, workspace=None, status=None, stream=None):
    """Places of the tokens' choices sorted by expert: slots [T][k], offsets [E + 1] where each expert's
    places begin, order [T k] the choice at each place (may be None)."""
    rc = (_dense._marshal or _dense._load()).expert_sort(ids, E, offsets, slots, order, workspace, status, _handle(stream))
    if rc:
        _fail("dlrm_expert_sort", rc)


def dlrm_dispatch_fwd(x, slots, xs, status=None, stream=None):
    """xs[slots[t][j]] = x[t]; rows of xs that no slot names stay as they were."""
    rc = (_dense._marshal or _dense._load()).dispatch_fwd(x, slots, xs, status, _handle(stream))
    if rc:
        _fail("dlrm_dispatch_fwd", rc)


def dlrm_dispatch_bwd(grad_xs, slots, grad_x, status=None, stream=None):
    """grad_x[t] = sum over j of grad_xs[slots[t][j]]."""
    rc = (_dense._marshal or _dense._load()).dispatch_bwd(grad_xs, slots, grad_x, status, _handle(stream))
    if rc:
        _fail("dlrm_dispatch_bwd", rc)


def dlrm_combine_fwd(ys, slots, probs, residual, y, status=None, stream=None):
    """y[t] = residual[t] + sum over j of probs[t][j] * ys[slots[t][j]]; residual may be None."""
    rc = (_dense._marshal or _dense._load()).combine_fwd(ys, slots, probs, residual, y, status, _handle(stream))
    if rc:
        _fail("dlrm_combine_fwd", rc)


def dlrm_combine_bwd(grad_y, ys, slots, probs, grad_ys, grad_probs, status=None, stream=None):
    """Gradients of ``dlrm_combine_fwd``; grad_ys or grad_probs may be None.  The residual's gradient is
    grad_y itself."""
    rc = (_dense._marshal or _dense._load()).combine_bwd(grad_y, ys, slots, probs, grad_ys, grad_probs, status, _handle(stream))
    if rc:
        _fail("dlrm_combine_bwd", rc)


def dlrm_pack8(x, q, exps, stream=None):
    """x in 8 bits: q [M][N] bytes, exps [M][ceil(N / 32)] the blocks' powers of two."""
    rc = (_dense._marshal or _dense._load()).pack8(x, q, exps, _handle(stream))
    if rc:
        _fail("dlrm_pack8", rc)


def dlrm_unpack8(q, exps, y, stream=None):
    """The values that q and exps stand for."""
    rc = (_dense._marshal or _dense._load()).unpack8(q, exps, y, _handle(stream))
    if rc:
        _fail("dlrm_unpack8", rc)


def dlrm_linear_bwd8_workspace_size(grad_y, x_q, w, act=DLRM_ACT_NONE, p=0.0) -> int:
    """Bytes for all three gradients; x_q may be None, as for a call without grad_w."""
    M, (N, K) = grad_y.shape[0], w.shape
    return _size("dlrm_linear_bwd8_workspace_size", *_at(grad_y), *_at(w), _code(w.dtype), M, N, K, act, p)


def dlrm_linear_bwd8(grad_y, x_q, x_exps, w, pre_q, pre_exps, grad_x, grad_w, grad_bias, act=DLRM_ACT_NONE, p=0.0, rng=None,
                     workspace=None, status=None, stream=None):
    """``dlrm_linear_bwd`` with the layer's input and pre-activation in 8 bits (``dlrm_pack8``)."""
    rc = (_dense._marshal or _dense._load()).linear_bwd8(grad_y, x_q, x_exps, w, pre_q, pre_exps, grad_x, grad_w, grad_bias,
                                                         act, p, rng, workspace, status, _handle(stream))
    if rc:
        _fail("dlrm_linear_bwd8", rc)
