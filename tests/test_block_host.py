"""Refusals of the residual blocks' entry points (include/dlrm_block.h): every call here fails a check
or has nothing to do, before any CUDA call; the binding's own checks; and the gradients' 64-bit formulas
against differences of the forward's."""

import ctypes
import os
import re

import pytest
import torch

import block_ref as ref
import dlrm_embeddings_dot_gb300 as dl
from dlrm_embeddings_dot_gb300 import build as libbuild
from test_dense_binding import Elsewhere, _never

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, ODD = 0x10000, 0x10001      # never dereferenced
OK, INVALID, UNSUPPORTED, WORKSPACE = dl.DLRM_OK, dl.DLRM_ERR_INVALID_ARG, dl.DLRM_ERR_UNSUPPORTED, dl.DLRM_ERR_WORKSPACE
BIG = 2**31 - 1


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return dl.load()


def test_constants_match_the_header():
    src = open(os.path.join(ROOT, "include", "dlrm_block.h")).read()
    found = dict(re.findall(r"\b(DLRM_(?:NORM|GATE)_[A-Z]+)\s*=\s*(\d+)", src) +
                 re.findall(r"#define\s+(DLRM_(?:BLOCK|ROUTE)_\w+)\s+(\d+)", src))
    assert len(found) == 8
    for n, v in found.items():
        assert getattr(dl, n) == int(v)


def _norm_fwd(L, y=FAKE, ldy=16, g=None, ldg=0, gc=16, res=FAKE, ldres=16, wp=None, bp=None, sc=None, w=None, b=None, dt=1,
              M=4, N=16, norm=0, act=0, eps=1e-6, r=FAKE, ldr=16, h=FAKE, ldh=16, st=FAKE):
    return L.dlrm_block_norm_fwd(y, ldy, g, ldg, gc, res, ldres, wp, bp, sc, w, b, dt, M, N, norm, act, eps, r, ldr, h, ldh, st,
                                 None)


def test_norm_forward_refusals(L):
    for kw in (dict(dt=3), dict(dt=-1), dict(M=-1), dict(N=0), dict(norm=2), dict(norm=-1), dict(act=3), dict(act=-1),
               dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")), dict(y=ODD), dict(ldy=15), dict(ldy=2**41),
               dict(res=ODD), dict(ldres=15), dict(r=None), dict(r=ODD), dict(ldr=15), dict(h=ODD), dict(ldh=15),
               dict(g=FAKE, ldg=15), dict(g=ODD, ldg=16), dict(g=FAKE, ldg=16, gc=8), dict(g=FAKE, ldg=16, gc=0),
               dict(wp=0x10002), dict(bp=ODD), dict(sc=ODD), dict(w=ODD), dict(b=ODD), dict(st=0x10004),
               dict(y=None), dict(y=None, r=None, g=FAKE, ldg=16), dict(y=None, r=None, wp=FAKE), dict(y=None, r=None, res=None),
               dict(y=None, r=None, bp=FAKE), dict(y=None, r=None, sc=FAKE), dict(y=None, r=None, h=None),
               dict(h=None, w=FAKE), dict(h=None, b=FAKE)):
        assert _norm_fwd(L, **kw) == INVALID, kw
        assert "dlrm_block_norm_fwd" in dl.dlrm_last_error()
    assert _norm_fwd(L, N=8193) == UNSUPPORTED and _norm_fwd(L, M=BIG) == UNSUPPORTED
    assert _norm_fwd(L, M=0) == OK and _norm_fwd(L, M=0, y=None, res=None, r=None, h=None) == OK


def _norm_bwd(L, gr=FAKE, ldgr=16, gh=FAKE, ldgh=16, y=FAKE, ldy=16, g=None, ldg=0, gc=16, r=FAKE, ldr=16, st=FAKE, wp=None,
              bp=None, sc=None, w=None, dt=1, M=4, N=16, norm=0, act=0, gy=FAKE, ldgy=16, gg=None, ldgg=0, gres=FAKE,
              ldgres=16, o=(None,) * 5, ws=None, wsb=0):
    return L.dlrm_block_norm_bwd(gr, ldgr, gh, ldgh, y, ldy, g, ldg, gc, r, ldr, st, wp, bp, sc, w, dt, M, N, norm, act, gy, ldgy,
                                 gg, ldgg, gres, ldgres, *o, ws, wsb, None)


def test_norm_backward_refusals(L):
    for kw in (dict(dt=3), dict(M=-1), dict(N=0), dict(norm=2), dict(act=3), dict(gr=ODD), dict(ldgr=15), dict(gh=ODD),
               dict(ldgh=15), dict(y=ODD), dict(ldy=15), dict(r=None), dict(r=ODD), dict(ldr=15), dict(st=None),
               dict(st=0x10004), dict(gy=ODD), dict(ldgy=15), dict(gres=ODD), dict(ldgres=15), dict(g=FAKE, ldg=15),
               dict(g=FAKE, ldg=16, gc=3), dict(gg=FAKE, ldgg=16), dict(g=FAKE, ldg=16, gg=FAKE, ldgg=15),
               dict(g=FAKE, ldg=16, gg=ODD, ldgg=16), dict(wp=ODD), dict(bp=ODD), dict(sc=ODD), dict(w=ODD),
               dict(gr=None, gh=None, r=None), dict(gh=None), dict(gh=None, r=None, w=FAKE),
               dict(gh=None, r=None, y=None, gy=None), dict(y=None), dict(y=None, gy=None, wp=FAKE), dict(y=None, gy=None, bp=FAKE),
               dict(y=None, gy=None, sc=FAKE), dict(y=None, gy=None, g=FAKE, ldg=16)):
        assert _norm_bwd(L, **kw) == INVALID, kw
        assert "dlrm_block_norm_bwd" in dl.dlrm_last_error()
    for i in range(5):
        one = [None] * 5
        one[i] = FAKE
        need = L.dlrm_block_norm_bwd_workspace_size(4, 16)
        assert need > 0
        assert _norm_bwd(L, o=one) == WORKSPACE and _norm_bwd(L, o=one, ws=FAKE, wsb=need - 1) == WORKSPACE
        assert _norm_bwd(L, o=one, ws=0x10080, wsb=need) == INVALID
        assert _norm_bwd(L, o=one, ws=None, wsb=need) == WORKSPACE
        odd = [None] * 5
        odd[i] = ODD
        assert _norm_bwd(L, o=odd, ws=FAKE, wsb=need) == INVALID
        side = dict(y=None, gy=None) if i < 3 else dict(gh=None, r=None)
        assert _norm_bwd(L, o=one, ws=FAKE, wsb=need, **side) == INVALID
    assert _norm_bwd(L, N=8193) == UNSUPPORTED and _norm_bwd(L, M=BIG) == UNSUPPORTED
    assert _norm_bwd(L, M=0) == OK and _norm_bwd(L, M=0, gr=None, gh=None, y=None) == OK
    size = L.dlrm_block_norm_bwd_workspace_size
    assert size(0, 16) == size(4, 0) == size(4, 8193) == size(-1, 4) == 0
    for N in (1, 255, 8192):   # 8192 needs no more than the documented growth: blocks times four rows of floats
        assert size(BIG - 2**20, N) % 256 == 0 and size(BIG - 2**20, N) <= 2 * 152 * 4 * (N + 7) * 4 + 255


def test_route_refusals(L):
    def fwd(l=FAKE, ld=16, dt=1, T=4, E=16, k=2, ids=FAKE, p=FAKE):
        return L.dlrm_route_fwd(l, ld, dt, T, E, k, ids, p, None)

    def bwd(gp=FAKE, ids=FAKE, p=FAKE, dt=1, T=4, E=16, k=2, gl=FAKE, ld=16):
        return L.dlrm_route_bwd(gp, ids, p, dt, T, E, k, gl, ld, None)

    for f, more in ((fwd, (dict(l=None), dict(l=ODD))), (bwd, (dict(gp=None), dict(gp=ODD), dict(gl=None), dict(gl=ODD)))):
        for kw in (dict(dt=3), dict(T=-1), dict(E=0), dict(k=0), dict(k=17), dict(ld=15), dict(ids=None), dict(ids=ODD),
                   dict(p=None), dict(p=ODD)) + more:
            assert f(**kw) == INVALID, kw
        for kw in (dict(E=257, ld=257), dict(k=9), dict(T=BIG)):
            assert f(**kw) == UNSUPPORTED, kw
        assert f(T=0) == OK and f(T=0, ids=None, p=None) == OK


def test_sort_refusals(L):
    def sort(ids=FAKE, T=4, k=2, E=16, off=FAKE, slots=FAKE, order=None, ws=None, wsb=0):
        return L.dlrm_expert_sort(ids, T, k, E, off, slots, order, ws, wsb, None, None)

    for kw in (dict(T=-1), dict(k=0), dict(E=0), dict(ids=None), dict(ids=ODD), dict(off=None), dict(off=ODD), dict(slots=None),
               dict(slots=ODD), dict(order=ODD)):
        assert sort(**kw) == INVALID, kw
    for kw in (dict(E=257), dict(k=9), dict(T=BIG), dict(T=2**28, k=8)):
        assert sort(**kw) == UNSUPPORTED, kw
    need = L.dlrm_expert_sort_workspace_size(50000, 2, 16)
    assert need > 0 and sort(T=50000) == WORKSPACE and sort(T=50000, ws=FAKE, wsb=need - 1) == WORKSPACE
    assert sort(T=50000, ws=0x10080, wsb=need) == INVALID
    assert L.dlrm_expert_sort_workspace_size(4, 9, 16) == L.dlrm_expert_sort_workspace_size(-1, 2, 16) == 0


def test_row_refusals(L):
    def disp(x=FAKE, ldx=16, s=FAKE, dt=1, T=4, k=2, H=16, R=8, xs=FAKE, ldxs=16):
        return L.dlrm_dispatch_fwd(x, ldx, s, dt, T, k, H, R, xs, ldxs, None, None)

    def back(x=FAKE, ldx=16, s=FAKE, dt=1, T=4, k=2, H=16, R=8, xs=FAKE, ldxs=16):
        return L.dlrm_dispatch_bwd(xs, ldxs, s, dt, T, k, H, R, x, ldx, None, None)

    def comb(x=FAKE, ldx=16, s=FAKE, dt=1, T=4, k=2, H=16, R=8, xs=FAKE, ldxs=16, p=FAKE, res=None, ldres=0):
        return L.dlrm_combine_fwd(xs, ldxs, s, p, res, ldres, dt, T, k, H, R, x, ldx, None, None)

    def cbwd(x=FAKE, ldx=16, s=FAKE, dt=1, T=4, k=2, H=16, R=8, xs=FAKE, ldxs=16, p=FAKE, ys=FAKE, ldys=16, gp=FAKE):
        return L.dlrm_combine_bwd(x, ldx, ys, ldys, s, p, dt, T, k, H, R, xs, ldxs, gp, None, None)

    for f, more in ((disp, ()), (back, ()), (comb, (dict(p=None), dict(p=ODD), dict(res=FAKE, ldres=15), dict(res=ODD, ldres=16))),
                    (cbwd, (dict(p=None), dict(p=ODD), dict(ys=None), dict(ys=ODD), dict(ldys=15), dict(gp=ODD),
                            dict(xs=None, gp=None)))):
        for kw in (dict(dt=3), dict(T=-1), dict(k=0), dict(H=0), dict(R=-1), dict(x=None), dict(x=ODD), dict(ldx=15),
                   dict(s=None), dict(s=ODD), dict(xs=ODD), dict(ldxs=15)) + more:
            assert f(**kw) == INVALID, (f.__name__, kw)
        if f is not cbwd:
            assert f(xs=None) == INVALID
        for kw in (dict(k=9), dict(T=BIG), dict(R=BIG), dict(H=BIG, ldx=2**31, ldxs=2**31)):
            assert f(**kw) == UNSUPPORTED, (f.__name__, kw)
        assert f(T=0) == OK and f(T=0, x=None, s=None, xs=None) == OK


def test_8_bit_refusals(L):
    def pack(x=FAKE, ldx=40, dt=1, M=4, N=40, q=ODD, ldq=40, e=ODD):
        return L.dlrm_pack8(x, ldx, dt, M, N, q, ldq, e, None)

    def unpack(x=FAKE, ldx=40, dt=1, M=4, N=40, q=ODD, ldq=40, e=ODD):
        return L.dlrm_unpack8(q, ldq, e, dt, M, N, x, ldx, None)

    for f in (pack, unpack):
        for kw in (dict(dt=3), dict(M=-1), dict(N=0), dict(x=None), dict(x=ODD), dict(ldx=39), dict(q=None), dict(ldq=39),
                   dict(e=None)):
            assert f(**kw) == INVALID, kw
        for kw in (dict(M=BIG), dict(N=BIG, ldx=2**31, ldq=2**31)):
            assert f(**kw) == UNSUPPORTED, kw
        assert f(M=0) == OK and f(M=0, x=None, q=None, e=None) == OK

    def bwd(g=FAKE, ldg=24, x=ODD, ldx=16, xe=ODD, w=FAKE, ldw=16, z=ODD, ldz=24, ze=ODD, dt=1, M=64, N=24, K=16, act=1, p=0.0,
            rng=None, dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE, wsb=1 << 30):
        return L.dlrm_linear_bwd8(g, ldg, x, ldx, xe, w, ldw, z, ldz, ze, dt, M, N, K, act, p, rng, dx, 16, dw, 16, db, ws, wsb,
                                  None, None)

    for kw in (dict(g=None), dict(g=ODD), dict(ldg=23), dict(x=None), dict(ldx=15), dict(xe=None), dict(w=None), dict(w=ODD),
               dict(z=None), dict(ldz=23), dict(ze=None), dict(dt=3), dict(M=-1), dict(N=0), dict(K=0), dict(act=4),
               dict(p=1.0), dict(p=0.1), dict(dx=ODD), dict(dw=ODD), dict(db=ODD), dict(ws=0x10080)):
        assert bwd(**kw) == INVALID, kw
        assert "dlrm_linear_bwd8" in dl.dlrm_last_error()
    assert bwd(M=BIG) == UNSUPPORTED
    for dt in (0, 1, 2):
        for M, N, K, act in ((64, 24, 16, 1), (64, 24, 16, 2), (5000, 8, 40, 0), (5000, 8, 40, 1)):
            need = L.dlrm_linear_bwd8_workspace_size(FAKE, N, FAKE, K, dt, M, N, K, act, 0.0)
            assert need > 0
            assert L.dlrm_linear_bwd8(FAKE, N, FAKE, K, FAKE, FAKE, K, FAKE, N, FAKE, dt, M, N, K, act, 0.0, None, FAKE, K, FAKE,
                                      K, FAKE, FAKE, need - 1, None, None) == WORKSPACE


# ------------------------------------------------------------------------------------------- binding
def _calls():
    """(name, function, arguments with every tensor given)"""
    f, i, u = torch.float32, torch.int32, torch.uint8

    def t(*s, dtype=f):
        return torch.zeros(*s, dtype=dtype)

    m, v = lambda: t(4, 16), lambda: t(16)
    k = lambda dtype: t(4, 2, dtype=dtype)
    ws, status = t(4096, dtype=u), t(1, dtype=i)
    return [
        (dl.dlrm_block_norm_fwd, dict(y=m(), gate=m(), residual=m(), w_post=v(), b_post=v(), scale=v(), w_pre=v(), b_pre=v(),
                                      r=m(), h=m(), stats=t(4, 4))),
        (dl.dlrm_block_norm_bwd, dict(grad_r=m(), grad_h=m(), y=m(), gate=m(), r=m(), stats=t(4, 4), w_post=v(), b_post=v(),
                                      scale=v(), w_pre=v(), grad_y=m(), grad_gate=m(), grad_residual=m(), grad_w_post=v(),
                                      grad_b_post=v(), grad_scale=v(), grad_w_pre=v(), grad_b_pre=v(), workspace=ws)),
        (dl.dlrm_route_fwd, dict(logits=m(), ids=k(i), probs=k(f))),
        (dl.dlrm_route_bwd, dict(grad_probs=k(f), ids=k(i), probs=k(f), grad_logits=m())),
        (dl.dlrm_expert_sort, dict(ids=k(i), E=3, offsets=t(4, dtype=i), slots=k(i), order=t(8, dtype=i), workspace=ws,
                                   status=status)),
        (dl.dlrm_dispatch_fwd, dict(x=m(), slots=k(i), xs=t(8, 16), status=status)),
        (dl.dlrm_dispatch_bwd, dict(grad_xs=t(8, 16), slots=k(i), grad_x=m(), status=status)),
        (dl.dlrm_combine_fwd, dict(ys=t(8, 16), slots=k(i), probs=k(f), residual=m(), y=m(), status=status)),
        (dl.dlrm_combine_bwd, dict(grad_y=m(), ys=t(8, 16), slots=k(i), probs=k(f), grad_ys=t(8, 16), grad_probs=k(f),
                                   status=status)),
        (dl.dlrm_pack8, dict(x=m(), q=t(4, 16, dtype=u), exps=t(4, 1, dtype=u))),
        (dl.dlrm_unpack8, dict(q=t(4, 16, dtype=u), exps=t(4, 1, dtype=u), y=m())),
        (dl.dlrm_linear_bwd8, dict(grad_y=t(4, 24), x_q=t(4, 16, dtype=u), x_exps=t(4, 1, dtype=u), w=t(24, 16),
                                   pre_q=t(4, 24, dtype=u), pre_exps=t(4, 1, dtype=u), grad_x=m(), grad_w=t(24, 16),
                                   grad_bias=t(24), act=1, p=0.1, rng=t(2, dtype=torch.int64), workspace=ws, status=status)),
    ]


CASES = [(i, name) for i, (_, a) in enumerate(_calls()) for name, v in a.items() if isinstance(v, torch.Tensor)]


def _on_device_0(call, args, want=99):
    """The call with a binding whose current device is 0 and whose entry points answer 99."""
    from dlrm_embeddings_dot_gb300 import block_abi, dense
    m = dense._load()
    at = ctypes.cast(_never, ctypes.c_void_p).value
    m.bind(dense._TYPES, lambda: 0, lambda d: 0, (at,) * 5)
    m.bind_block(torch.uint8, (at,) * len(block_abi.ENTRY_POINTS))
    try:
        call(**args)
    finally:
        dense._marshal = None
        dense._load()


def _there(args, device=0):
    return {k: Elsewhere(v, device) if isinstance(v, torch.Tensor) else v for k, v in args.items()}


@pytest.mark.parametrize("i", range(len(_calls())))
def test_right_calls_reach_the_entry_points(i):
    libbuild.build()
    call, args = _calls()[i]
    with pytest.raises(dl.DlrmError, match="returned 99"):
        _on_device_0(call, _there(args))


@pytest.mark.parametrize("i,name", CASES)
def test_tensors_elsewhere_are_refused(i, name):
    """On the host, on another device, of another type, of another size, with a column stride."""
    call, args = _calls()[i]
    t = args[name]
    for other, error, text in (
            (Elsewhere(t, -1), ValueError, f"^{name} is not on a CUDA device"),
            (Elsewhere(t, 1), ValueError, f"^{name} is on device 1, not on the current one"),
            (Elsewhere(t.double(), 0), TypeError, None),
            (Elsewhere(torch.zeros(*t.shape, 1, dtype=t.dtype), 0), ValueError, None),
            (Elsewhere(torch.zeros(*(s + 1 for s in t.shape), dtype=t.dtype), 0), ValueError, None),
            (Elsewhere(torch.zeros(*t.shape, 2, dtype=t.dtype)[..., 0], 0), ValueError, None)):
        if error is TypeError and name in ("workspace", "status"):
            continue            # any type that has the bytes
        if text is None and error is ValueError and name in ("workspace", "status"):
            continue
        a = _there(args)
        a[name] = other
        with pytest.raises(error, match=text):
            _on_device_0(call, a)


def test_codes_past_32_bits_are_refused():
    call, args = _calls()[0]
    for name in ("norm", "gate_act"):
        with pytest.raises(ValueError, match=f"^{name} is"):
            _on_device_0(call, dict(_there(args), **{name: 2**32}))
    call, args = _calls()[4]
    with pytest.raises(ValueError, match="^E is"):
        _on_device_0(call, dict(_there(args), E=2**32 + 3))


def test_missing_tensors_are_refused():
    for i, names in ((0, ("y", "residual")), (1, ("grad_r", "grad_h")), (8, ("ys", "grad_ys"))):
        call, args = _calls()[i]
        with pytest.raises(ValueError):
            _on_device_0(call, dict(_there(args), **{n: None for n in names}))


# ------------------------------------------------------------------------------------------- formulas
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("gate,per_row", [("raw", False), ("sigmoid", False), ("silu", False), ("silu", True)])
def test_norm_gradients_against_differences(layer, gate, per_row):
    """Central differences of the forward's formula in 64 bits, h = 2^-10: truncation below h^2 times the
    third derivative (some ten for values of order 1), 1e-4 of the directional derivative's terms."""
    gen = torch.Generator().manual_seed(1)
    M, N, eps = 5, 12, 1e-3

    def rand(*s):
        return torch.randn(*s, generator=gen, dtype=torch.float64)

    a = dict(y=rand(M, N), g=rand(M, 1 if per_row else N), res=rand(M, N), w_post=rand(N), b_post=rand(N), scale=rand(N),
             w_pre=rand(N), b_pre=rand(N))
    cr, ch = rand(M, N), rand(M, N)

    def loss(**v):
        o = ref.forward(*v.values(), layer, gate, eps)
        return float((o["r"][0] * cr).sum() + (o["h"][0] * ch).sum())

    o = ref.forward(*a.values(), layer, gate, eps)
    stats = torch.cat([*o["y_stats"], *o["r_stats"]], 1)
    grads = ref.backward(cr, ch, a["y"], a["g"], o["r"][0], stats, a["w_post"], a["b_post"], a["scale"], a["w_pre"], layer, gate)
    for name, key in (("y", "y"), ("g", "gate"), ("res", "residual"), ("w_post", "w_post"), ("b_post", "b_post"),
                      ("scale", "scale"), ("w_pre", "w_pre"), ("b_pre", "b_pre")):
        v, h = rand(*a[name].shape), 2.0**-10
        quotient = (loss(**dict(a, **{name: a[name] + h * v})) - loss(**dict(a, **{name: a[name] - h * v}))) / (2 * h)
        terms = grads[key][0] * v
        assert abs(quotient - float(terms.sum())) <= 1e-4 * float(terms.abs().sum()), name


def test_published_values_of_the_8_bit_floats():
    v = ref.code_values()
    assert v[0x7e] == 448 and v[0x01] == 2.0**-9 and v[0x08] == 2.0**-6 and v[0x38] == 1 and v[0xb8] == -1 and v[127].isnan()
    q, e = ref.pack8(torch.tensor([[448.0, 1.0, 2.0**-9, 0.0, -17.0, 19.0, -0.0] + [0.0] * 25 + [896.0, 1.0]]))
    assert e.tolist() == [[127, 128]] and q[0, :7].tolist() == [0x7e, 0x38, 1, 0, 0xd8, 0x5a, 0x80] and q[0, 33] == 0x30
