"""What the dense layer's gradient holds between its two halves, against 64-bit forms: dZ is not
rounded to a 2-byte type, and what dropout's scale or a slope takes past fp16's range is not lost.

Bounds (u = half an ulp of the output type; A = the same expression on absolute values):
  * a' of NONE and RELU is 0 or 1 and dropout's scale is applied to the sums: dZ is exact, and so is
    its plane; the sums' error is (L + 8) 2^-23 A, the scale's and the last rounding's 2^-23 and u
  * GELU and SILU: the slope is within 2^-20 of its largest size, 1.2; the value in two terms within
    2^-16 (bf16) or 2^-20 (fp16) of itself, fp16's second term on a grid of 2^-24
"""

import pytest
import torch

import dense_ref as ref
from gpu_util import dev

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
TERMS = {"f16": 2.0**-20, "bf16": 2.0**-16, "f32": 0.0}


def _rand(g, *shape, std=1.0, dtype="f32"):
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * std).to(ref.TYPES[dtype]).to(dev())


def _gradients(dl, dy, x, w, z, name, p=0.0, seed=(5, 6)):
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(w.shape[0], device=dev())
    n = dl.dlrm_linear_bwd_workspace_size(dy, x, w, act=ref.ACT[name], p=p)
    ws = torch.empty(n, dtype=torch.uint8, device=dev()) if n else None
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    dl.dlrm_linear_bwd(dy, x, w, z, dx, dw, db, act=ref.ACT[name], p=p, workspace=ws, status=status,
                       rng=torch.tensor(seed, dtype=torch.int64, device=dev()))
    assert int(status.item()) == 0
    return dx, dw, db


def _want(dy, x, w, z, name, dtype, p=0.0, seed=(5, 6)):
    """{gradient: (value, bound)} in 64 bits on the GPU."""
    dy, x, w = dy.double(), x.double(), w.double()
    (M, K), N = x.shape, w.shape[0]
    scale = 1.0
    g = dy
    if p:
        kept, scale = ref.keep_scale(*seed, M, N, p)
        g = torch.where(kept.to(dev()), dy, torch.zeros_like(dy))
    dz = g if name == "none" else g * ref.slope(z.double(), name)
    if name in ("none", "relu"):
        one = torch.zeros_like(dz)
    else:
        one = 2.0**-20 * 1.2 * g.abs() + TERMS[dtype] * dz.abs() + (2.0**-25 if dtype == "f16" else 0.0)
    size = dz.abs() + one

    def product(a, b, ea, L):
        v, e = a @ b * scale, (ea @ b.abs() + (L + 8) * 2.0**-23 * (size_of(a) @ b.abs())) * scale
        return v, e + 2.0**-22 * v.abs()

    def size_of(a):
        return size if a.shape == size.shape and a is dz else size.t()

    return {"dx": product(dz, w, one, N), "dw": product(dz.t(), x, one.t(), M),
            "db": (dz.sum(0) * scale, (one.sum(0) + (M + 16) * 2.0**-23 * size.sum(0)) * scale)}


# tiles and few outputs, split K and not, aligned and ragged
SIZES = [(256, 512, 1024), (700, 40, 264), (65, 48, 72), (130, 77, 129), (3000, 24, 40), (256, 16, 1024), (40, 5, 333),
         (9000, 1, 72)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("name,p", [("none", 0.3), ("relu", 0.1), ("gelu", 0.0), ("silu", 0.2)])
def test_gradient_has_one_rounding(cuda_lib, dtype, M, N, K, name, p):
    g = torch.Generator().manual_seed(M + N + K)
    x, w = _rand(g, M, K, dtype=dtype), _rand(g, N, K, std=K**-0.5, dtype=dtype)
    dy, z = _rand(g, M, N, std=0.1, dtype=dtype), _rand(g, M, N, dtype=dtype)
    got = _gradients(cuda_lib, dy, x, w, z, name, p)
    want = _want(dy, x, w, z, name, dtype, p)
    for t, k in zip(got, ("dx", "dw", "db")):
        ref.assert_close(t, *want[k], "f32" if k == "db" else dtype, k)


@pytest.mark.parametrize("M,N,K", [(130, 40, 72), (130, 40, 77), (130, 8, 72), (130, 8, 77)])
@pytest.mark.parametrize("name,p", [("none", 0.5), ("relu", 0.75), ("gelu", 0.5), ("silu", 0.0)])
def test_gradient_past_the_range_of_fp16(cuda_lib, M, N, K, name, p):
    """|dY| up to 65,504 with a slope above 1 or a scale of 2 and 4: dZ does not fit fp16, the gradients do."""
    g = torch.Generator().manual_seed(M + N)
    x, w = _rand(g, M, K, std=2.0**-12, dtype="f16"), _rand(g, N, K, std=2.0**-12, dtype="f16")
    dy = (torch.rand(M, N, generator=g, dtype=torch.float64) * 15504 + 50000).half().to(dev())
    z = (torch.rand(M, N, generator=g, dtype=torch.float64) + 1.5).half().to(dev())   # slopes up to 1.13
    got = _gradients(cuda_lib, dy, x, w, z, name, p)
    want = _want(dy, x, w, z, name, "f16", p)
    for t, k in zip(got, ("dx", "dw", "db")):
        assert bool(torch.isfinite(t).all()), k
        ref.assert_close(t, *want[k], "f32" if k == "db" else "f16", k)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("N", [40, 8])
@pytest.mark.parametrize("name", ["none", "gelu", "silu"])
def test_infinite_and_nan_gradients(cuda_lib, dtype, N, name):
    """An infinity in dY reaches its row of dX and its column's row of dW with the sign 32 bits give, a
    NaN as NaN, and nothing else."""
    M, K = 130, 72
    g = torch.Generator().manual_seed(N)
    x, w = _rand(g, M, K, dtype=dtype), _rand(g, N, K, std=K**-0.5, dtype=dtype)
    dy, z = _rand(g, M, N, std=0.1, dtype=dtype), _rand(g, M, N, dtype=dtype)
    dy[3, 2], dy[9, 5] = -INF, NAN
    dx, dw, db = _gradients(cuda_lib, dy, x, w, z, name)
    dz = dy.double() if name == "none" else dy.double() * ref.slope(z.double(), name)
    for got, want in ((dx, dz @ w.double()), (dw, dz.t() @ x.double()), (db, dz.sum(0))):
        got = got.double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        inf = torch.isinf(want)
        assert int(inf.sum()) > 0 and torch.equal(got[inf], want[inf])
        assert bool(torch.isfinite(got[torch.isfinite(want)]).all())


def _plain32(z, name, slope):
    """The header's definition in 32 bits by torch."""
    if name == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * 0.5**0.5))
        return cdf + z * torch.exp(-0.5 * z * z) / (2 * torch.pi) ** 0.5 if slope else z * cdf
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s)) if slope else z / (1 + torch.exp(-z))


@pytest.mark.parametrize("N", [1, 24])
@pytest.mark.parametrize("name", ["gelu", "silu"])
@pytest.mark.parametrize("span", [0.5, 3.0, 8.0])
def test_fp32_activations_are_as_exact_as_their_definition_in_32_bits(cuda_lib, name, span, N):
    """The same formula in the same arithmetic has the same error: the root mean square over a range is
    that of torch's form to within a quarter.  (x is z, the weight 1: the sum before is exact.)"""
    M = 1 << 16
    z = torch.linspace(-span, span, M, device=dev())
    x, w = z[:, None].contiguous(), torch.zeros(N, 1, device=dev())
    w[0] = 1.0
    y = torch.empty(M, N, device=dev())
    n = cuda_lib.dlrm_linear_fwd_workspace_size(x, w)
    cuda_lib.dlrm_linear_fwd(x, w, None, None, y, act=ref.ACT[name],
                             workspace=torch.empty(n, dtype=torch.uint8, device=dev()) if n else None)
    dy, pre = torch.zeros(M, N, device=dev()), torch.zeros(M, N, device=dev())
    dy[:, 0], pre[:, 0] = 1.0, z
    dx, _, _ = _gradients(cuda_lib, dy, x, w, pre, name)
    for got, form, exact in ((y[:, 0], _plain32(z, name, False), ref.act(z.double(), name)),
                             (dx[:, 0], _plain32(z, name, True), ref.slope(z.double(), name))):
        own, plain = ((t.double() - exact).square().mean().sqrt().item() for t in (got, form))
        assert own <= 1.25 * plain, (own, plain)


def _rms_share(got, exact):
    return ((got.double() - exact).norm() / exact.norm()).item()


@pytest.mark.parametrize("M,N,K", [(32, 4096, 4096), (9, 1024, 480), (64, 512, 1000), (32768, 16, 256), (20000, 9, 300)])
def test_fp32_sums_on_fragments_are_fp32_sums(cuda_lib, M, N, K):
    """Few rows or few outputs, more than eight tokens: blocks of 16 of K, each within 2^-22 for the cuts of its
    six sums, are added in fp32, a rounding of 2^-24 each; for terms of random sign they add like their
    square root."""
    g = torch.Generator().manual_seed(M)
    x, w = _rand(g, M, K), _rand(g, N, K, std=K**-0.5)
    y = torch.empty(M, N, device=dev())
    n = cuda_lib.dlrm_linear_fwd_workspace_size(x, w)
    cuda_lib.dlrm_linear_fwd(x, w, None, None, y, workspace=torch.empty(n, dtype=torch.uint8, device=dev()) if n else None)
    assert _rms_share(y, x.double() @ w.double().t()) <= (K / 16) ** 0.5 * 2.0**-24 + 2.0**-22


@pytest.mark.parametrize("H,I", [(2048, 1024), (1001, 515)])
def test_fp32_mixture_sums_are_fp32_sums(cuda_lib, H, I):
    """One expert with 32 tokens: both products within the same bound."""
    T = 32
    g = torch.Generator().manual_seed(H)
    x, wr = _rand(g, T, H), torch.zeros(1, H, device=dev())
    w1, w2 = _rand(g, 1, I, H, std=H**-0.5), _rand(g, 1, H, I, std=I**-0.5)
    y, probs, ids = torch.empty_like(x), torch.empty(T, 1, device=dev()), torch.empty(T, 1, dtype=torch.int32, device=dev())
    cuda_lib.dlrm_moe_fwd(x, wr, w1, w2, None, y, ids, probs, act=0, gated=False, workspace=torch.empty(
        cuda_lib.dlrm_moe_fwd_workspace_size(x, wr, w1, w2, 1), dtype=torch.uint8, device=dev()))
    exact = x.double() @ w1[0].double().t() @ w2[0].double().t()
    assert _rms_share(y, exact) <= ((H / 16) ** 0.5 + (I / 16) ** 0.5) * 2.0**-24 + 2 * 2.0**-22


@pytest.mark.parametrize("M,N,K", [(8192, 1024, 512), (8192, 1024, 1024), (2000, 520, 2048), (8192, 512, 4096), (4099, 771, 771),
                                   (300, 96, 1100), (20000, 40, 1048)])
def test_fp32_sums_of_any_length_are_fp32_sums(cuda_lib, M, N, K):
    """384 of K are added up on the tensor cores, 24 sums that are each cut by half of 2^-23 on average, at
    sizes that grow like a square root (two thirds of the last): 24 / 2 * 2 / 3 * 2^-23 = 9.5e-7, less where the
    accumulator keeps bits below; beyond, such blocks are added in fp32.  So no length has more than a
    library's fp32 product of 2,048 of K, 8e-7."""
    g = torch.Generator().manual_seed(K)
    x, w = _rand(g, M, K), _rand(g, N, K, std=K**-0.5)
    y = torch.empty(M, N, device=dev())
    n = cuda_lib.dlrm_linear_fwd_workspace_size(x, w)
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    cuda_lib.dlrm_linear_fwd(x, w, None, None, y, status=status,
                             workspace=torch.empty(n, dtype=torch.uint8, device=dev()) if n else None)
    assert _rms_share(y, x.double() @ w.double().t()) <= 8e-7 and int(status.item()) == 0
    # the gradients sum over N and over M
    dy, dx, dw, db = _rand(g, M, N), torch.empty_like(x), torch.empty_like(w), torch.empty(N, device=dev())
    n = cuda_lib.dlrm_linear_bwd_workspace_size(dy, x, w)
    cuda_lib.dlrm_linear_bwd(dy, x, w, None, dx, dw, db, workspace=torch.empty(n, dtype=torch.uint8, device=dev()))
    assert _rms_share(dx, dy.double() @ w.double()) <= 8e-7
    assert _rms_share(dw, dy.double().t() @ x.double()) <= 8e-7


@pytest.mark.parametrize("M,N,K", [(16384, 512, 1024), (9000, 515, 771)])
def test_long_fp32_sums_repeat_and_give_up(cuda_lib, M, N, K):
    """Sums in segments have the same bits in every call, and a wait that gives up among them ends the call
    with DLRM_STATUS_TIMEOUT, the next one being right."""
    g = torch.Generator().manual_seed(N)
    x, w, r, b = _rand(g, M, K), _rand(g, N, K, std=K**-0.5), _rand(g, M, N), _rand(g, N)
    n = cuda_lib.dlrm_linear_fwd_workspace_size(x, w)
    ws = torch.empty(n, dtype=torch.uint8, device=dev())
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    outs = [torch.empty(M, N, device=dev()) for _ in range(4)]
    for y in outs[:3]:
        cuda_lib.dlrm_linear_fwd(x, w, b, r, y, act=2, workspace=ws, status=status)
    assert int(status.item()) == 0 and torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    try:
        cuda_lib.dlrm_set_wait_limit(0)
        cuda_lib.dlrm_linear_fwd(x, w, b, r, outs[3], act=2, workspace=ws, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == cuda_lib.DLRM_STATUS_TIMEOUT
    finally:
        cuda_lib.dlrm_set_wait_limit(-1)
    status.zero_()
    cuda_lib.dlrm_linear_fwd(x, w, b, r, outs[3], act=2, workspace=ws, status=status)
    assert int(status.item()) == 0 and torch.equal(outs[0], outs[3])


@pytest.mark.parametrize("limit", [0, 300, 3000, 30000])
@pytest.mark.parametrize("M,N,K,dtype", [(8192, 1024, 480, "f16"), (300, 200, 264, "bf16"), (9000, 515, 771, "f32"),
                                         (16384, 512, 1024, "f32"), (2048, 512, 512, "bf16")])
def test_a_layer_given_up_anywhere_leaves_the_next_one_right(cuda_lib, M, N, K, dtype, limit):
    """Waits that give up at the start, or after some cycles in the middle of a tile: the call ends, says so if
    it did, and the forward and the gradient after it have their bits."""
    g = torch.Generator().manual_seed(limit)
    x, w, dy = _rand(g, M, K, dtype=dtype), _rand(g, N, K, std=K**-0.5, dtype=dtype), _rand(g, M, N, dtype=dtype)
    wf = torch.empty(max(1, cuda_lib.dlrm_linear_fwd_workspace_size(x, w)), dtype=torch.uint8, device=dev())
    wb = torch.empty(max(1, cuda_lib.dlrm_linear_bwd_workspace_size(dy, x, w, act=2)), dtype=torch.uint8, device=dev())
    status = torch.zeros(1, dtype=torch.int32, device=dev())

    def run():
        y, dx, dw, db = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(w), torch.empty(N, device=dev())
        cuda_lib.dlrm_linear_fwd(x, w, None, None, y, act=2, workspace=wf, status=status)
        cuda_lib.dlrm_linear_bwd(dy, x, w, dy, dx, dw, db, act=2, workspace=wb, status=status)
        torch.cuda.synchronize()
        return y, dx, dw, db

    want = run()
    assert int(status.item()) == 0
    for _ in range(4):
        try:
            cuda_lib.dlrm_set_wait_limit(limit)
            run()
        finally:
            cuda_lib.dlrm_set_wait_limit(-1)
        assert int(status.item()) in ((cuda_lib.DLRM_STATUS_TIMEOUT,) if limit == 0 else (0, cuda_lib.DLRM_STATUS_TIMEOUT))
        status.zero_()
        assert all(torch.equal(a, b) for a, b in zip(run(), want)) and int(status.item()) == 0
