"""Refusals of the dense network's entry points (include/dlrm_dense.h): every call here fails a
check or has nothing to do, before any CUDA call; and the binding's own checks of its tensors."""

import ctypes
import os
import re

import pytest
import torch

import dense_ref as ref
import dlrm_embeddings_dot_gb300 as dl
from dlrm_embeddings_dot_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, ODD = 0x10000, 0x10001      # never dereferenced
OK, INVALID, UNSUPPORTED, WORKSPACE = dl.DLRM_OK, dl.DLRM_ERR_INVALID_ARG, dl.DLRM_ERR_UNSUPPORTED, dl.DLRM_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return dl.load()


def test_constants_match_the_header():
    src = open(os.path.join(ROOT, "include", "dlrm_dense.h")).read()
    found = dict(re.findall(r"\b(DLRM_ACT_[A-Z]+)\s*=\s*(\d+)", src) + re.findall(r"#define\s+(DLRM_MOE_\w+)\s+(\d+)", src))
    assert len(found) == 7
    for n, v in found.items():
        assert getattr(dl, n) == int(v)


def test_published_answers_of_the_generator():
    assert ref.philox([0, 0, 0, 0], [0, 0]) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    n = ref.numbers(2**63 + 7, 2**40 + 1, 3, 20)
    for r, c in ((0, 0), (1, 9), (2, 19)):
        w = ref.philox([c // 8, r, 1, 2**8], [7, 2**31])[(c % 8) // 2]
        assert n[r, c] == (w >> 16 * (c % 2)) & 0xFFFF


def _dropout(L, x=FAKE, ldx=8, r=None, ldr=0, dt=0, M=4, N=8, p=0.1, rng=FAKE, y=FAKE, ldy=8):
    return L.dlrm_dropout_fwd(x, ldx, r, ldr, dt, M, N, p, rng, y, ldy, None)


def test_dropout_refusals(L):
    for kw in (dict(x=None), dict(y=None), dict(dt=3), dict(dt=-1), dict(M=-1), dict(N=0), dict(p=-0.1), dict(p=1.0),
               dict(p=float("nan")), dict(p=1 - 2.0**-18), dict(rng=None), dict(rng=0x10004), dict(ldx=7), dict(ldy=7),
               dict(r=FAKE, ldr=7), dict(x=ODD), dict(y=ODD), dict(r=ODD, ldr=8), dict(ldx=2**41)):
        assert _dropout(L, **kw) == INVALID, kw
        assert "dlrm_dropout_fwd" in dl.dlrm_last_error()
    assert _dropout(L, M=0) == OK and _dropout(L, M=0, x=None, y=None) == OK
    assert _dropout(L, M=0, p=2.0) == INVALID
    assert L.dlrm_dropout_bwd(None, 8, 0, 4, 8, 0.1, FAKE, FAKE, 8, None) == INVALID
    assert "dlrm_dropout_bwd" in dl.dlrm_last_error()


def _fwd(L, x=FAKE, ldx=16, w=FAKE, ldw=16, b=None, r=None, ldr=0, dt=1, M=4, N=8, K=16, act=0, p=0.0, rng=None, y=FAKE,
         ldy=8, pre=None, ldp=0, ws=None, wsb=0):
    return L.dlrm_linear_fwd(x, ldx, w, ldw, b, r, ldr, dt, M, N, K, act, p, rng, y, ldy, pre, ldp, ws, wsb, None, None)


def test_linear_fwd_refusals(L):
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(dt=3), dict(M=-1), dict(N=0), dict(K=0), dict(act=4),
               dict(act=-1), dict(p=1.0), dict(p=0.1), dict(ldx=15), dict(ldw=15), dict(ldy=7), dict(x=ODD), dict(w=ODD),
               dict(y=ODD), dict(b=0x10002), dict(r=FAKE, ldr=7), dict(r=ODD, ldr=8), dict(pre=FAKE, ldp=7),
               dict(pre=ODD, ldp=8)):
        assert _fwd(L, **kw) == INVALID, kw
        assert "dlrm_linear_fwd" in dl.dlrm_last_error()
    for big in (dict(M=2**31 - 1), dict(N=2**31 - 1, ldy=2**31), dict(K=2**31 - 1, ldx=2**31, ldw=2**31)):
        assert _fwd(L, **big) == UNSUPPORTED, big
    assert _fwd(L, M=0) == OK and _fwd(L, M=0, x=None, y=None, w=None) == OK


def test_linear_workspace_refusals(L):
    sizes = {}
    for dt in (0, 1, 2):
        for M, N, K in ((4, 8, 16), (4, 24, 16), (1000, 40, 13), (5000, 520, 264), (5000, 8, 16)):
            need = L.dlrm_linear_fwd_workspace_size(FAKE, K, FAKE, K, dt, M, N, K)
            sizes[dt, M, K] = need
            if need:
                assert _fwd(L, dt=dt, M=M, N=N, K=K, ldx=K, ldw=K, ldy=N) == WORKSPACE
                assert _fwd(L, dt=dt, M=M, N=N, K=K, ldx=K, ldw=K, ldy=N, ws=FAKE, wsb=need - 1) == WORKSPACE
                assert _fwd(L, dt=dt, M=M, N=N, K=K, ldx=K, ldw=K, ldy=N, ws=FAKE + 16, wsb=need) == INVALID
            need = L.dlrm_linear_bwd_workspace_size(FAKE, N, FAKE, K, FAKE, K, dt, M, N, K, 1, 0.1)
            assert need > 0 or (M, N) == (4, 8)   # a few rows of few outputs are one chunk
            if need:
                assert _bwd(L, dt=dt, M=M, N=N, K=K, ws=FAKE, wsb=need - 1) == WORKSPACE
                assert _bwd(L, dt=dt, M=M, N=N, K=K, ws=None, wsb=need) == WORKSPACE
    for bad in ((3, 4, 8, 16), (1, -1, 8, 16), (1, 4, 0, 16), (1, 4, 8, 0), (1, 0, 8, 16)):
        assert L.dlrm_linear_fwd_workspace_size(FAKE, 16, FAKE, 16, *bad) == 0
        assert L.dlrm_linear_bwd_workspace_size(FAKE, 16, FAKE, 16, FAKE, 16, *bad, 1, 0.1) == 0


def _bwd(L, g=FAKE, x=FAKE, w=FAKE, pre=FAKE, dt=1, M=4, N=8, K=16, act=1, p=0.1, rng=FAKE, dx=FAKE, dw=FAKE, db=FAKE,
         ws=FAKE, wsb=1 << 40, ldg=None, ldx=None, ldw=None, ldp=None, lddx=None, lddw=None):
    return L.dlrm_linear_bwd(g, ldg or N, x, ldx or K, w, ldw or K, pre, ldp or N, dt, M, N, K, act, p, rng, dx, lddx or K,
                             dw, lddw or K, db, ws, wsb, None, None)


def test_linear_bwd_refusals(L):
    for kw in (dict(g=None), dict(x=None), dict(w=None), dict(pre=None), dict(dt=3), dict(M=-1), dict(N=0), dict(K=0),
               dict(act=4), dict(p=1.5), dict(rng=None), dict(g=ODD), dict(x=ODD), dict(w=ODD), dict(pre=ODD),
               dict(dx=ODD), dict(dw=ODD), dict(db=0x10002), dict(ldg=7), dict(ldx=15), dict(ldw=15), dict(ldp=7),
               dict(lddx=15), dict(lddw=15), dict(ws=FAKE + 8, N=24)):
        assert _bwd(L, **kw) == INVALID, kw
    assert _bwd(L, M=0, dw=None, db=None) == OK       # nothing to write


def _moe(L, x=FAKE, ldx=16, wr=FAKE, w1=FAKE, w2=FAKE, r=None, ldr=0, dt=1, T=4, H=16, I=8, E=4, k=2, act=3, gated=1,
         y=FAKE, ldy=16, ids=FAKE, probs=FAKE, ws=FAKE, wsb=1 << 40):
    return L.dlrm_moe_fwd(x, ldx, wr, w1, w2, r, ldr, dt, T, H, I, E, k, act, gated, y, ldy, ids, probs, ws, wsb, None, None)


def test_moe_refusals(L):
    for kw in (dict(x=None), dict(wr=None), dict(w1=None), dict(w2=None), dict(y=None), dict(ids=None), dict(probs=None),
               dict(dt=3), dict(T=-1), dict(H=0), dict(I=0), dict(E=0), dict(k=0), dict(k=5), dict(act=4), dict(ldx=15),
               dict(ldy=15), dict(r=FAKE, ldr=15), dict(x=ODD), dict(w2=ODD), dict(ids=0x10002), dict(ws=FAKE + 8)):
        assert _moe(L, **kw) == INVALID, kw
    for kw in (dict(T=65), dict(E=257), dict(E=16, k=9)):
        assert _moe(L, **kw) == UNSUPPORTED, kw
    need = L.dlrm_moe_fwd_workspace_size(1, 4, 16, 8, 4, 2)
    assert need > 0 and _moe(L, wsb=need - 1) == WORKSPACE and _moe(L, ws=None) == WORKSPACE
    assert _moe(L, T=0, x=None) == OK
    assert L.dlrm_moe_fwd_workspace_size(1, 0, 16, 8, 4, 2) == 0 and L.dlrm_moe_fwd_workspace_size(1, 4, 16, 8, 4, 5) == 0


def test_existing_calls_still_refuse_bf16(L):
    assert L.dlrm_emb_fwd(FAKE, 2, FAKE, 1, 16, 2, FAKE, FAKE, 2, FAKE, 0, None, None) == INVALID
    assert L.dlrm_interact_fwd(FAKE, FAKE, 2, 2, 16, 2, FAKE, 64, None, None) == INVALID


def test_binding_checks_its_tensors():
    x, w, y = torch.zeros(4, 16), torch.zeros(8, 16), torch.zeros(4, 8)
    with pytest.raises(TypeError):
        dl.dlrm_linear_fwd(x, w.half(), None, None, y)
    with pytest.raises(TypeError):
        dl.dlrm_linear_fwd(x.double(), w.double(), None, None, y.double())
    with pytest.raises(TypeError):
        dl.dlrm_linear_fwd(x, w, torch.zeros(8).half(), None, y)
    with pytest.raises(ValueError):
        dl.dlrm_linear_fwd(x, torch.zeros(8, 15), None, None, y)
    with pytest.raises(ValueError):
        dl.dlrm_linear_fwd(torch.zeros(16, 4).t(), w, None, None, y)
    with pytest.raises(ValueError):
        dl.dlrm_linear_fwd(x, w, None, None, torch.zeros(4, 9))
    with pytest.raises(ValueError):
        dl.dlrm_dropout_fwd(x, torch.zeros(4, 15), torch.zeros(4, 16), 0.1, None)
    with pytest.raises(TypeError):
        dl.dlrm_dropout_fwd(x, None, torch.zeros(4, 16), 0.1, torch.zeros(2))
    with pytest.raises(ValueError):
        dl.dlrm_moe_fwd(x, torch.zeros(3, 16), torch.zeros(3, 8, 16), torch.zeros(3, 16, 8), None, torch.zeros(4, 16),
                        torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), gated=True)
