"""Rows of the residual blocks' matrices (include/dlrm_block.h) that lie more than 2^32 bytes apart, in every layout
of the kernels: to the bit what the same rows give next to each other."""

import pytest
import torch

import dense_ref as dref
from gpu_util import dev

pytestmark = pytest.mark.gpu

FAR = 2**31 + 72          # 2-byte elements from row to row
ROOM = 3 * 2**14          # columns of all matrices of a test together


@pytest.fixture(scope="module")
def base():
    return torch.empty(2 * FAR + ROOM, dtype=torch.float16, device=dev())


class Far:
    """Matrices of three rows in one buffer, one after another in its columns."""

    def __init__(self, base, dtype, lead):
        self.base, self.at = base.view(dref.TYPES[dtype]) if dtype in dref.TYPES else base.view(torch.uint8), lead

    def __call__(self, N, like=None):
        e = self.base.element_size()
        v = self.base.as_strided((3, N), (FAR * 2 // e if e < 4 else FAR // 2, 1), self.at)
        self.at += (N + 63) // 32 * 32
        assert self.at * e <= ROOM * 2
        return v if like is None else v.copy_(like)


def _near(t, lead):
    """A copy with its rows next to each other, on the 16-byte grid where Far's are."""
    N = t.shape[1]
    return torch.empty(3, (lead + N + 63) // 32 * 32, dtype=t.dtype, device=dev())[:, lead:lead + N].copy_(t)


def _rand(g, N, dtype, std=1.0):
    return (torch.randn(3, N, generator=g) * std).to(dref.TYPES[dtype]).to(dev())


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("lead", [0, 1])
@pytest.mark.parametrize("N", [64, 520, 1024, 771])
def test_norms(cuda_lib, base, dtype, lead, N):
    g = torch.Generator().manual_seed(N)
    far = Far(base, dtype, lead)
    near = {n: _rand(g, N, dtype) for n in ("y", "gate", "residual", "gr", "gh")}
    v = [torch.rand(N, generator=g).to(dev()) for _ in range(5)]
    results = []
    for put in (lambda t: _near(t, lead), lambda t: far(N, t)):
        a = {n: put(t) for n, t in near.items()}
        o = [put(torch.full_like(near["y"], 7.0)) for _ in range(5)]
        st, gv = torch.empty(3, 4, device=dev()), torch.empty(5, N, device=dev())
        ws = torch.empty(cuda_lib.dlrm_block_norm_bwd_workspace_size(a["y"]), dtype=torch.uint8, device=dev())
        kw = dict(norm=1, gate_act=1)
        cuda_lib.dlrm_block_norm_fwd(a["y"], a["gate"], a["residual"], *v, o[0], o[1], st, **kw)
        cuda_lib.dlrm_block_norm_bwd(a["gr"], a["gh"], a["y"], a["gate"], o[0], st, *v[:4], *o[2:], *gv.unbind(0), workspace=ws, **kw)
        results.append([t.clone() for t in (*o, st, gv)])
    assert all(torch.equal(p, q) for p, q in zip(*results))


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("lead", [0, 1])
@pytest.mark.parametrize("H", [40, 520, 1024, 771])
def test_rows_of_experts(cuda_lib, base, dtype, lead, H):
    g = torch.Generator().manual_seed(H)
    far = Far(base, dtype, lead)
    slots = torch.tensor([[2], [-1], [0]], dtype=torch.int32, device=dev())
    probs = torch.tensor([[0.5], [0.25], [2.0]], device=dev())
    x, ys, res = (_rand(g, H, dtype) for _ in range(3))
    results = []
    for put in (lambda t: _near(t, lead), lambda t: far(H, t)):
        a, b, c = put(x), put(ys), put(res)
        xs, y, gx, gys = (put(torch.full_like(x, 7.0)) for _ in range(4))
        gp = torch.empty(3, 1, device=dev())
        cuda_lib.dlrm_dispatch_fwd(a, slots, xs)
        cuda_lib.dlrm_combine_fwd(b, slots, probs, c, y)
        cuda_lib.dlrm_dispatch_bwd(b, slots, gx)
        cuda_lib.dlrm_combine_bwd(a, b, slots, probs, gys, gp)
        results.append([t.clone() for t in (xs, y, gx, gys, gp)])
    assert all(torch.equal(p, q) for p, q in zip(*results))


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("lead", [0, 1])
@pytest.mark.parametrize("N,K", [(24, 64), (8, 520), (33, 65), (1, 771)])
def test_8_bits(cuda_lib, base, dtype, lead, N, K):
    """The matrices in 8 bits far apart, then those of the layer's gradient that go with them."""
    g = torch.Generator().manual_seed(N + K)
    x, z, dy, w = _rand(g, K, dtype), _rand(g, N, dtype), _rand(g, N, dtype, 0.1), _rand(g, K, dtype)[:1].repeat(N, 1)
    u8 = dict(dtype=torch.uint8, device=dev())
    results = []
    for place in (False, True):
        far, bits = Far(base, dtype, lead), Far(base, "bytes", 2 * ROOM - 8192 + lead)
        put = (lambda t: far(t.shape[1], t)) if place else (lambda t: _near(t, lead))
        code = bits if place else (lambda n: _near(torch.empty(3, n, **u8), lead))
        X, Z = put(x), put(z)
        xq, zq, xe, ze = code(K), code(N), torch.empty(3, -(-K // 32), **u8), torch.empty(3, -(-N // 32), **u8)
        cuda_lib.dlrm_pack8(X, xq, xe)
        cuda_lib.dlrm_pack8(Z, zq, ze)
        back, dx = put(torch.full_like(x, 7.0)), put(torch.full_like(x, 7.0))
        cuda_lib.dlrm_unpack8(xq, xe, back)
        dw, db, d = torch.empty_like(w), torch.empty(N, device=dev()), put(dy)
        n = cuda_lib.dlrm_linear_bwd8_workspace_size(d, xq, w, act=2)
        cuda_lib.dlrm_linear_bwd8(d, xq, xe, w, zq, ze, dx, dw, db, act=2,
                                  workspace=torch.empty(n, dtype=torch.uint8, device=dev()) if n else None)
        results.append([t.clone() for t in (xq, zq, xe, ze, back, dx, dw, db)])
    assert all(torch.equal(p, q) for p, q in zip(*results))
