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


# probs * h in two scaled fp16 values or three bf16 ones is within 2^-21 of itself or of the run's
# largest; ref.moe's bound for any other u than fp16's has no term for fp16's least values
FINE = 2.0**-21


def _scaled_case(T, H, I, E, dtype, x_std, w1_std, w2_std, seed, lead=0):
    x, wr, w1, w2 = _case(T, H, I, E, dtype, True, lead, seed)
    # activations of the size x_std * w1_std with weights in their type's ordinary range
    x.mul_(x_std)
    wr.div_(x_std)
    w1.mul_(w1_std)
    w2.mul_(w2_std)
    return x, wr, w1, w2


@pytest.mark.parametrize("T,H,I,E,k,lead", [(3, 64, 136, 4, 2, 0), (20, 256, 512, 6, 3, 0), (64, 64, 48, 2, 2, 0),
                                            (5, 67, 35, 5, 2, 0), (33, 64, 64, 3, 1, 1)])
@pytest.mark.parametrize("x_std,w1_std,w2_std", [(64.0, 16.0, 2.0**-14), (2.0**-10, 1.0, 2.0**10)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_moe_activations_of_any_size(cuda_lib, dtype, T, H, I, E, k, lead, x_std, w1_std, w2_std):
    """Gated products around 2^20, past fp16's range, against small w2; and around 2^-20, below its
    normal range, against large ones: y is as exact as with activations around 1."""
    x, wr, w1, w2 = _scaled_case(T, H, I, E, dtype, x_std, w1_std, w2_std, 5, lead)
    y, ids, probs, ws = _buffers(cuda_lib, x, wr, w1, w2, k)
    cuda_lib.dlrm_moe_fwd(x, wr, w1, w2, None, y, ids, probs, act=3, gated=True, workspace=ws)
    d = [t.double().cpu() for t in (x, wr, w1, w2)]
    wy, ey, _, _ = ref.moe(*d, None, ids.cpu().long(), "silu", True, FINE)
    assert bool(torch.isfinite(y).all())
    ref.assert_close(y, wy, ey, dtype, "y")


def test_moe_runs_of_different_size(cuda_lib):
    """Runs of 16 hidden values whose sizes differ by 2^40 within a token, and between the tokens of an expert."""
    T, H, I = 9, 16, 1024
    g = torch.Generator().manual_seed(3)
    size = 2.0 ** ((torch.arange(I) // 16 * 7) % 41 - 20.0)
    x = (torch.randn(T, H, generator=g, dtype=torch.float64) * 2.0 ** (torch.arange(T)[:, None] % 3 * 2.0)).half().to(dev())
    w1 = torch.randn(1, I, H, generator=g, dtype=torch.float64)
    # size carried by w1 as far as fp16 goes, by both factors of a gated product
    w1 = torch.cat([w1 * size[:, None].clamp(2.0**-10, 2.0**10), torch.randn(1, I, H, generator=g, dtype=torch.float64) *
                    (size / size.clamp(2.0**-10, 2.0**10))[:, None]], 1).half().to(dev())
    w2 = (torch.randn(1, H, I, generator=g, dtype=torch.float64) * 2.0**-14).half().to(dev())
    wr = torch.zeros(1, H, dtype=torch.float16, device=dev())
    y, ids, probs, ws = _buffers(cuda_lib, x, wr, w1, w2, 1)
    cuda_lib.dlrm_moe_fwd(x, wr, w1, w2, None, y, ids, probs, act=0, gated=True, workspace=ws)
    d = [t.double().cpu() for t in (x, wr, w1, w2)]
    wy, ey, _, _ = ref.moe(*d, None, ids.cpu().long(), "none", True, FINE)
    # some sums pass fp16's range themselves (65,520 and more round to an infinity)
    far, near = wy.abs() - ey > 65520, wy.abs() + ey < 65520
    assert int(near.sum()) > 60 and torch.equal(y.double().cpu()[far], wy[far].sign() * float("inf"))
    ref.assert_close(y.cpu()[near], wy[near], ey[near], "f16", "y")


@pytest.mark.parametrize("H,I", [(64, 136), (67, 35)])
def test_moe_tokens_do_not_change_one_another(cuda_lib, H, I):
    """fp16: a token whose activations leave fp16's range gives the other tokens of its experts the same bits."""
    T, E, k = 9, 2, 2
    x, wr, w1, w2 = _case(T, H, I, E, "f16", True, seed=4)
    w2[:, 0].mul_(0.0)     # an output that stays in range for the large token
    outs = []
    for size in (1.0, 1024.0, 2.0**-12):
        x2 = x.clone()
        x2[4].mul_(size)
        y, ids, probs, ws = _buffers(cuda_lib, x2, wr, w1, w2, k)
        cuda_lib.dlrm_moe_fwd(x2, wr, w1, w2, None, y, ids, probs, act=0, gated=True, workspace=ws)
        outs.append(y)
    keep = [t for t in range(T) if t != 4]
    assert torch.equal(outs[1][keep], outs[0][keep]) and torch.equal(outs[2][keep], outs[0][keep])
    assert not bool(torch.isnan(outs[1]).any()) and bool(torch.isfinite(outs[1][4, :1]).all())


@pytest.mark.parametrize("H", [8, 9])
def test_moe_bf16_hidden_values_have_24_bits(cuda_lib, H):
    """y = h0 - h1 with h0 and h1 apart by 2^-21 of themselves, every sum exact in fp32."""
    a, b, c = 1 + 2.0**-7, 2.0**-12 * (1 + 2.0**-7), 2.0**-21
    t = torch.bfloat16
    x, w1, w2 = torch.zeros(1, H, dtype=t), torch.zeros(1, H, H, dtype=t), torch.zeros(1, H, H, dtype=t)
    x[0, :3] = 1.0
    w1[0, 0, :3], w1[0, 1, :3] = torch.tensor([a, b, c]).to(t), torch.tensor([a, b, 0.0]).to(t)
    w2[0, 0, 0], w2[0, 0, 1] = 1.0, -1.0
    x, w1, w2, wr = x.to(dev()), w1.to(dev()), w2.to(dev()), torch.zeros(1, H, dtype=t, device=dev())
    y, ids, probs, ws = _buffers(cuda_lib, x, wr, w1, w2, 1)
    cuda_lib.dlrm_moe_fwd(x, wr, w1, w2, None, y, ids, probs, act=0, gated=False, workspace=ws)
    assert y[0].tolist() == [c] + [0.0] * (H - 1)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_moe_infinite_and_nan_activations(cuda_lib, dtype):
    """A token with an infinity or a NaN gives what 32 bits give (act none, gated: the product of two
    infinities or of infinities and numbers), and the others what they give without it."""
    T, H, I, E = 6, 32, 48, 1
    x, wr, w1, w2 = _case(T, H, I, E, dtype, True, seed=8)
    clean = _buffers(cuda_lib, x, wr, w1, w2, 1)
    wr.zero_()
    cuda_lib.dlrm_moe_fwd(x, wr, w1, w2, None, clean[0], clean[1], clean[2], act=0, gated=True, workspace=clean[3])
    x2 = x.clone()
    x2[1, 4], x2[4, 7] = float("nan"), float("inf")
    w1[0, :, 7].abs_()
    w1[0, :, 7].add_(0.125)
    w1c = w1.clone()
    got = _buffers(cuda_lib, x, wr, w1, w2, 1)
    cuda_lib.dlrm_moe_fwd(x, wr, w1c, w2, None, clean[0], clean[1], clean[2], act=0, gated=True, workspace=clean[3])
    wr[0, 0] = 0.0
    cuda_lib.dlrm_moe_fwd(x2, wr, w1c, w2, None, got[0], got[1], got[2], act=0, gated=True, workspace=got[3])
    y = got[0].cpu()
    # one expert: its probability is exp(NaN) where the logit is 0 * inf or 0 * NaN, so NaN for both tokens
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[4]).all())
    for t in (0, 2, 3, 5):
        assert torch.equal(got[0][t], clean[0][t])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("limit", [0, 300, 3000, 30000])
def test_a_mixture_given_up_anywhere_leaves_the_next_one_right(cuda_lib, dtype, limit):
    T, H, I, E, k = 12, 2048, 512, 16, 4
    x, wr, w1, w2 = _case(T, H, I, E, dtype, True)
    status = torch.zeros(1, dtype=torch.int32, device=dev())

    def run():
        y, ids, probs, ws = _buffers(cuda_lib, x, wr, w1, w2, k)
        cuda_lib.dlrm_moe_fwd(x, wr, w1, w2, None, y, ids, probs, workspace=ws, status=status)
        torch.cuda.synchronize()
        return y, ids, probs

    want = run()
    assert int(status.item()) == 0
    for _ in range(4):
        try:
            cuda_lib.dlrm_set_wait_limit(limit)
            run()
        finally:
            cuda_lib.dlrm_set_wait_limit(-1)
        assert int(status.item()) in (0, cuda_lib.DLRM_STATUS_TIMEOUT)
        status.zero_()
        assert all(torch.equal(a, b) for a, b in zip(run(), want)) and int(status.item()) == 0
