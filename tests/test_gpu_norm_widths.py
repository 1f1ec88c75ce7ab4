"""The residual blocks' norms (include/dlrm_block.h) at every number of warps a row takes, on the 16-byte grid and off
it, with rows enough that each group of warps goes round its ring of rows several times; the kept statistics to their
own bounds; and the gradients against 64-bit autograd.

Rows repeat with a period of 61, which no number of groups on a GPU is a multiple of, so a row that is
taken from another's place is a wrong one: the first 61 are compared with the 64-bit form, the others with
the first by their bits (what a row gets does not depend on where it is)."""

import pytest
import torch

import block_ref as ref
import dense_ref as dref
from gpu_util import dev
from test_gpu_block import _codes, _d, _empty, _guard_ok, _rand, _ws

pytestmark = pytest.mark.gpu

DTYPES = ["f32", "f16", "bf16"]
PERIOD = 61
GRID = [256, 512, 768, 1024, 1280, 1536, 1792, 2048, 2560, 2816, 3200, 4096, 5000, 5120, 6144, 8192]     # 1 .. 32 warps
ANY = [200, 257, 515, 771, 1025, 1285, 1541, 1799, 2049, 2817, 3201, 4095, 4999, 6143, 8189]
WIDTHS = [(n, 0, 0) for n in GRID] + [(n, 0, 0) for n in ANY] + [(2048, 8, 0), (768, 0, 1), (4096, 3, 0)]
# centred with everything; RMS, a gate by row; block alone; next norm alone
OPTIONS = [(True, "silu", False, True, True, True, True), (False, "sigmoid", True, True, True, False, True),
           (True, "raw", False, True, False, True, True), (True, None, False, False, True, True, True)]


def _rows(N):
    """Ten rows of every group of 24 warps an SM, 152 SMs, or 61 where those are fewer; a multiple of 61."""
    return -(-10 * 152 * 24 // -(-N // 256) // PERIOD) * PERIOD


def _case(N, pad, lead, dtype, option):
    """(inputs of all rows, the first 61 rows' in 64 bits)"""
    layer, gate, per_row, post, pre, vectors, residual = option
    g = torch.Generator().manual_seed(N)
    M = _rows(N)

    def matrix(cols, **kw):
        few = _rand(g, PERIOD, cols, dtype=dtype, **kw)
        out = _empty(M, cols, dtype, pad, lead)
        out.copy_(few.repeat(M // PERIOD, 1))
        return out

    v = lambda mean: _rand(g, N, std=0.3, mean=mean)
    a = dict(y=matrix(N, std=1.5, mean=0.2) if post else None,
             gate=matrix(1 if per_row else N, mean=0.3) if gate else None, residual=matrix(N, std=2.0, mean=-0.1),
             w_post=v(1.0) if post else None, b_post=v(0.0) if post and vectors else None, scale=v(0.5) if post and vectors else None,
             w_pre=v(1.0) if pre else None, b_pre=v(0.0) if pre and vectors else None)
    return M, a, {k: _d(t[:PERIOD]) if t is not None and t.dim() == 2 else _d(t) for k, t in a.items()}


def _repeats(t):
    """All rows have the bits of the first 61."""
    b = t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16).view(-1, PERIOD, t.shape[1])
    return bool((b == b[:1]).all())


def _stat_bounds(v, e, layer, eps):
    """Of the mean, and of 1 / sqrt relative to it: block_ref.norm's for rows v known to e."""
    n = v.shape[1]
    m = v.mean(1, keepdim=True) if layer else 0 * v[:, :1]
    em = e.mean(1, keepdim=True) + (n + 8) * ref.SUM * v.abs().mean(1, keepdim=True) if layer else 0 * m
    d, ed = v - m, e + em + ref.OP * (v.abs() + m.abs())
    ss = (d * d).mean(1, keepdim=True)
    return em, ((2 * d.abs() * ed + ed * ed).mean(1, keepdim=True) + (n + 8) * ref.SUM * ss) / (ss + eps) + ref.OP


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("option", OPTIONS)
@pytest.mark.parametrize("N,pad,lead", WIDTHS)
def test_norm_rows_in_turn(cuda_lib, dtype, option, N, pad, lead):
    layer, gate, per_row, post, pre, vectors, residual = option
    eps = 1e-5
    M, a, few = _case(N, pad, lead, dtype, option)
    r, h = (_empty(M, N, dtype, pad, lead) if on else None for on in (post, pre))
    st = torch.full((M, 4), 7.0, device=dev())
    cuda_lib.dlrm_block_norm_fwd(a["y"], a["gate"], a["residual"], a["w_post"], a["b_post"], a["scale"], a["w_pre"], a["b_pre"], r,
                                 h, st, eps=eps, **_codes(cuda_lib, option))
    want = ref.forward(few["y"], few["gate"], few["residual"], few["w_post"], few["b_post"], few["scale"], few["w_pre"],
                       few["b_pre"], layer, gate or "raw", eps, pre)
    for name, got in (("r", r), ("h", h)):
        if got is not None:
            dref.assert_close(got[:PERIOD], *want[name], dtype, name)
            assert _repeats(got) and _guard_ok(got), name
    assert _repeats(st)
    zero = torch.zeros(PERIOD, N, dtype=torch.float64)
    if post:
        em, rel = _stat_bounds(few["y"], zero, layer, eps)
        dref.assert_close(st[:PERIOD, 0:1], want["y_stats"][0], em, "f32", "mean of y")
        dref.assert_close(st[:PERIOD, 1:2], want["y_stats"][1], rel * want["y_stats"][1], "f32", "1 / sqrt of y")
    if pre:      # of r before its rounding, whatever the type
        em, rel = _stat_bounds(*(want["r"] if post else (few["residual"], zero)), layer, eps)
        dref.assert_close(st[:PERIOD, 2:3], want["r_stats"][0], em, "f32", "mean of r")
        dref.assert_close(st[:PERIOD, 3:4], want["r_stats"][1], rel * want["r_stats"][1], "f32", "1 / sqrt of r")
    # its gradient, from these statistics
    g = torch.Generator().manual_seed(N + 1)
    gr, gh = (torch.empty_like(a["residual"]) for _ in range(2))
    for t in (gr, gh):
        t.copy_(_rand(g, PERIOD, N, std=0.1, dtype=dtype).repeat(M // PERIOD, 1))
    gh = gh if pre else None
    out = {"residual": _empty(M, N, dtype, pad, lead)}
    vec = lambda: torch.full((N,), 7.0, device=dev())
    if post:
        out.update(y=_empty(M, N, dtype, pad, lead), w_post=vec(), b_post=vec(), scale=vec())
        if gate:
            out["gate"] = _empty(M, 1 if per_row else N, dtype, pad, lead)
    if pre:
        out.update(w_pre=vec(), b_pre=vec())
    kept = (r if post else a["residual"]) if pre else None
    cuda_lib.dlrm_block_norm_bwd(gr, gh, a["y"], a["gate"], kept, st, a["w_post"], a["b_post"], a["scale"], a["w_pre"],
                                 *(out.get(k) for k in ("y", "gate", "residual", "w_post", "b_post", "scale", "w_pre", "b_pre")),
                                 workspace=_ws(cuda_lib.dlrm_block_norm_bwd_workspace_size(gr)), **_codes(cuda_lib, option))
    part = lambda t: None if t is None else _d(t[:PERIOD])
    want = ref.backward(part(gr), part(gh), few["y"], few["gate"], part(kept), part(st), few["w_post"], few["b_post"],
                        few["scale"], few["w_pre"], layer, gate or "raw")
    for k, got in out.items():
        v, bound = want[k]
        if got.dim() == 1:     # the same rows M / 61 times; the sum's length is M's
            times = M // PERIOD
            dref.assert_close(got, v * times, bound * times * (M + 8) / (PERIOD + 8), "f32", k)
        else:
            dref.assert_close(got[:PERIOD], v, bound, dtype, k)
            assert _repeats(got) and _guard_ok(got), k


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("gate,per_row", [(None, False), ("raw", False), ("sigmoid", True), ("silu", False)])
@pytest.mark.parametrize("M,N", [(37, 72), (50, 300), (33, 1030), (12, 2504)])
def test_norm_gradient_against_autograd(cuda_lib, layer, gate, per_row, M, N):
    """fp32, statistics in 64 bits rounded to 32 and r to fp32, none of them the kernel's own.  The longest chain sums N
    terms of the norm before the next block, N of that after the block and M rows, each to (L + 8) 2^-23 of its terms'
    sizes, which cancel to a tenth at most: in all within (2 N + M + 50) 2^-23 * 10 of the gradient's
    largest value."""
    g = torch.Generator().manual_seed(M * N)
    rand = lambda *s, std=1.0, mean=0.0: _rand(g, *s, std=std, mean=mean)
    a = dict(y=rand(M, N, std=1.5, mean=0.2), gate=rand(M, 1 if per_row else N, mean=0.3) if gate else None,
             residual=rand(M, N, std=2.0, mean=-0.1), w_post=rand(N, std=0.3, mean=1.0), b_post=rand(N, std=0.3),
             scale=rand(N, std=0.3, mean=0.5), w_pre=rand(N, std=0.3, mean=1.0), b_pre=rand(N, std=0.3))
    cr, ch, eps = rand(M, N, std=0.1), rand(M, N, std=0.1), 1e-5
    leaf = {k: _d(v).requires_grad_() for k, v in a.items() if v is not None}

    def norm(v):
        m = v.mean(1, keepdim=True) if layer else torch.zeros_like(v[:, :1])
        s = 1 / torch.sqrt(((v - m) ** 2).mean(1, keepdim=True) + eps)
        return (v - m) * s, m, s

    x, m0, s0 = norm(leaf["y"])
    q = 1.0 if gate is None else ref.gate(leaf["gate"], gate)
    r = leaf["residual"] + leaf["scale"] * q * (x * leaf["w_post"] + leaf["b_post"])
    x, m1, s1 = norm(r)
    h = x * leaf["w_pre"] + leaf["b_pre"]
    ((r * _d(cr)).sum() + (h * _d(ch)).sum()).backward()
    st = torch.cat((m0, s0, m1, s1), 1).detach().float().to(dev())
    out = {k: torch.full_like(v, 7.0) for k, v in a.items() if v is not None}
    cuda_lib.dlrm_block_norm_bwd(cr, ch, a["y"], a["gate"], r.detach().float().to(dev()), st, a["w_post"], a["b_post"], a["scale"],
                                 a["w_pre"], *(out.get(k) for k in ("y", "gate", "residual", "w_post", "b_post", "scale", "w_pre", "b_pre")),
                                 workspace=_ws(cuda_lib.dlrm_block_norm_bwd_workspace_size(cr)), norm=int(layer),
                                 gate_act=ref.GATES[gate or "raw"])
    for k, got in out.items():
        want = leaf[k].grad
        assert float((_d(got) - want).abs().max()) <= (2 * N + M + 50) * 2.0**-23 * 10 * float(want.abs().max()), k
