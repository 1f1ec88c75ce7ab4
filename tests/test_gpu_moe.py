"""The mixture-of-experts layer off the 16-byte grid and in the ways programs run it, against the
64-bit form of ``dense_ref``."""

import pytest
import torch

import dense_ref as ref
from gpu_util import dev

pytestmark = pytest.mark.gpu


def _case(T, H, I, E, dtype, gated, lead=0, seed=0):
    """x, w_router, w1, w2 on the device; lead: elements before each one's first."""
    g = torch.Generator().manual_seed(seed + T * 1000 + H)

    def make(std, *shape):
        n = 1
        for s in shape:
            n *= s
        flat = torch.empty(n + lead, dtype=ref.TYPES[dtype], device=dev())
        t = flat[lead:].view(*shape)
        t.copy_(torch.randn(*shape, generator=g, dtype=torch.float64) * std)
        return t

    return (make(1.0, T, H), make(H**-0.5, E, H), make(H**-0.5, E, I * (2 if gated else 1), H), make(I**-0.5, E, H, I))


def _buffers(dl, x, wr, w1, w2, k):
    T = x.shape[0]
    ws = torch.empty(dl.dlrm_moe_fwd_workspace_size(x, wr, w1, w2, k), dtype=torch.uint8, device=dev())
    return torch.empty_like(x), torch.full((T, k), -1, dtype=torch.int32, device=dev()), torch.empty(T, k, device=dev()), ws


def _check(x, wr, w1, w2, res, k, name, gated, dtype, y, ids, probs):
    d = [None if t is None else t.double().cpu() for t in (x, wr, w1, w2, res)]
    logits = d[0] @ d[1].t()
    want, _ = ref.moe_route(logits, k)
    near = (x.shape[1] + 8) * 2.0**-22 * (d[0].abs() @ d[1].abs().t()).max()
    got = ids.cpu().long()
    assert bool(((torch.gather(logits, 1, got) - torch.gather(logits, 1, want)).abs() <= near).all())
    assert all(len(set(r)) == k for r in got.tolist())
    wy, ey, wp, ep = ref.moe(*d, got, name, gated, ref.U[dtype] if dtype != "f32" else 0.0)
    ref.assert_close(probs, wp, ep, "f32", "probs")
    ref.assert_close(y, wy, ey, dtype, "y")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,H,I,E,k,name,gated,lead", [
    (40, 1001, 515, 40, 6, "silu", True, 0),      # widths off the grid; logits shared out by clusters; K over several stages
    (64, 777, 131, 200, 8, "relu", False, 0),     # more logits than partial tiles
    (3, 2050, 33, 24, 2, "gelu", True, 0),        # a unit's K split between warps
    (20, 512, 256, 16, 4, "silu", True, 1),       # aligned widths, misaligned bases
    (1, 1024, 512, 8, 2, "gelu", False, 1)])
def test_moe_off_the_grid(cuda_lib, dtype, T, H, I, E, k, name, gated, lead):
    x, wr, w1, w2 = _case(T, H, I, E, dtype, gated, lead)
    res = x.clone() if T % 2 == 0 else None
    y, ids, probs, ws = _buffers(cuda_lib, x, wr, w1, w2, k)
    cuda_lib.dlrm_moe_fwd(x, wr, w1, w2, res, y, ids, probs, act=ref.ACT[name], gated=gated, workspace=ws)
    _check(x, wr, w1, w2, res, k, name, gated, dtype, y, ids, probs)
