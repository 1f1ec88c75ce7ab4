"""The dense network on the GPU (include/dlrm_dense.h) against plain 64-bit forms
(``dense_ref``, which also derives the error bounds): dense layer forward and backward,
dropout, and the mixture-of-experts layer for a few tokens."""

import itertools

import numpy as np
import pytest
import torch

import dense_ref as ref
from gpu_util import dev

pytestmark = pytest.mark.gpu

DTYPES = ["f32", "f16", "bf16"]
NAN, INF = float("nan"), float("inf")


def _rand(g, *shape, std=1.0, dtype="f32", pad=0, lead=0):
    """Normal values on the device; pad: extra columns between rows; lead: elements before the first."""
    t = torch.randn(*shape[:-1], shape[-1] + pad + lead, generator=g, dtype=torch.float64) * std
    return t.to(ref.TYPES[dtype]).to(dev())[..., lead:lead + shape[-1]]


def _rng(seed, offset):
    def wrap(v):
        return v - 2**64 if v >= 2**63 else v
    return torch.tensor([wrap(seed), wrap(offset)], dtype=torch.int64, device=dev())


def _empty(M, N, dtype, pad=0):
    """Output with pad guard columns that must stay as they are."""
    return torch.full((M, N + pad), 7.0, dtype=ref.TYPES[dtype], device=dev())[:, :N]


def _guard_ok(t):
    base = t._base if t._base is not None else t
    return bool((base[:, t.shape[1]:] == 7.0).all())


def _ws(n):
    return torch.empty(n, dtype=torch.uint8, device=dev()) if n else None


def _d(t):
    return None if t is None else t.double().cpu()


# ------------------------------------------------------------------------------------------- dropout
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,pad", [(1, 1, 0), (1, 8, 0), (3, 7, 0), (5, 24, 8), (37, 129, 0), (64, 480, 3),
                                     (513, 40, 0), (2, 4099, 0)])
@pytest.mark.parametrize("p,residual", [(0.1, False), (0.5, True), (0.0, True), (1e-6, False), (0.99, True)])
def test_dropout(cuda_lib, dtype, M, N, pad, p, residual):
    g = torch.Generator().manual_seed(M * N)
    x = _rand(g, M, N, dtype=dtype, pad=pad)
    r = _rand(g, M, N, dtype=dtype, pad=pad) if residual else None
    seed, offset = 2**63 + 12345, 2**40 + 3
    y = _empty(M, N, dtype, pad=5)
    cuda_lib.dlrm_dropout_fwd(x, r, y, p, _rng(seed, offset))
    kept, scale = ref.keep_scale(seed, offset, M, N, p)
    want = torch.where(kept, _d(x) * scale, torch.zeros(M, N, dtype=torch.float64))
    if residual:
        want = want + _d(r)
    # the scaling and the sum round in fp32
    ref.assert_close(y, want, 2.0**-23 * (want.abs() + scale * _d(x).abs()), dtype, "dropout")
    assert _guard_ok(y)
    if not residual:
        gx = torch.empty_like(y)
        cuda_lib.dlrm_dropout_bwd(x, gx, p, _rng(seed, offset))
        assert torch.equal(gx, y), "the backward's mask differs from the forward's"


def test_generator_known_answers(cuda_lib):
    """The published known answers of Philox4x32-10 come out of the kernel: with key and counter 0
    the words are 6627e8d5 e169c58d bc57ac4c 9b00dbd8; the thresholds around each number decide."""
    words = ref.philox([0, 0, 0, 0], [0, 0])
    assert words == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    nums = [v for w in words for v in (w & 0xFFFF, w >> 16)]
    assert ref.numbers(0, 0, 1, 8)[0].tolist() == nums
    x = torch.ones(1, 8, device=dev())
    y = torch.empty_like(x)
    for i, v in enumerate(nums):
        for t, kept in ((v, True), (v + 1, False)):
            cuda_lib.dlrm_dropout_fwd(x, None, y, t / 65536, _rng(0, 0))
            assert (y[0, i].item() != 0) == kept


def test_dropout_drops_infinities_and_nan(cuda_lib):
    x = torch.tensor([[INF, -INF, NAN, 1.0] * 64], device=dev())
    y = torch.empty_like(x)
    cuda_lib.dlrm_dropout_fwd(x, None, y, 0.5, _rng(5, 6))
    kept = ref.keep_scale(5, 6, 1, 256, 0.5)[0][0]
    out = y.cpu()[0]
    assert bool((out[~kept] == 0).all()) and 64 < int(kept.sum()) < 192
    assert torch.equal(torch.isnan(out[kept]), torch.isnan(x.cpu()[0][kept]))


def test_dropout_rate_and_independence(cuda_lib):
    """A million elements: the kept share within five standard deviations of the rate in force, the
    masks of another offset, another seed and a neighbouring row agree no more than chance."""
    M, N, p = 1024, 1024, 0.3
    x = torch.ones(M, N, dtype=torch.float16, device=dev())
    ys = []
    for rng in ((1, 0), (1, 1), (2, 0)):
        y = torch.empty_like(x)
        cuda_lib.dlrm_dropout_fwd(x, None, y, p, _rng(*rng))
        ys.append((y != 0).cpu())
    q = 1 - ref.threshold(p) / 65536
    n = M * N
    assert abs(ys[0].double().mean().item() - q) < 5 * (q * (1 - q) / n) ** 0.5
    same = q * q + (1 - q) ** 2
    for other in (ys[1], ys[2], ys[0].roll(1, 0), ys[0].roll(1, 1)):
        assert abs((ys[0] == other).double().mean().item() - same) < 5 * (same * (1 - same) / n) ** 0.5


def test_dropout_past_32_bits(cuda_lib):
    """Element positions past 2^32: the last row and column of 2^21 + 3 rows of 2,056 columns."""
    M, N = 2**21 + 3, 2056
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    x = torch.ones(M, N, dtype=torch.float16, device=dev())
    y = torch.empty_like(x)
    cuda_lib.dlrm_dropout_fwd(x, None, y, 0.25, _rng(9, 1))
    tail = y[-2:].cpu()
    for i, row in enumerate((M - 2, M - 1)):
        for col in (0, 5, N - 1):
            w = ref.philox([col // 8, row, 1, 0], [9, 0])[(col % 8) // 2]
            kept = (w >> 16 * (col % 2) & 0xFFFF) >= ref.threshold(0.25)
            assert (tail[i, col].item() != 0) == kept
    assert abs((y != 0).float().mean(1).mean().item() - 0.75) < 1e-3


# ------------------------------------------------------------------------------------------- dense layer
SIZES = [(1, 1, 1), (1, 1024, 480), (2, 17, 13), (7, 64, 64), (8, 256, 128), (9, 33, 300), (16, 16, 1), (24, 1, 256),
         (33, 130, 65), (64, 512, 1024), (65, 48, 72), (127, 255, 129), (128, 128, 64), (129, 257, 200), (300, 1, 40),
         (257, 520, 520), (1000, 96, 13), (640, 384, 448)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("name,p,bias,residual,pre,pad", [
    ("none", 0.0, False, False, False, 0), ("relu", 0.1, True, False, False, 0), ("gelu", 0.0, True, True, True, 8),
    ("silu", 0.3, True, True, True, 3)])
def test_linear_fwd(cuda_lib, dtype, M, N, K, name, p, bias, residual, pre, pad):
    g = torch.Generator().manual_seed(M + 31 * N + 977 * K)
    x = _rand(g, M, K, dtype=dtype, pad=pad)
    w = _rand(g, N, K, std=K**-0.5, dtype=dtype, pad=pad)
    b = _rand(g, N) if bias else None
    r = _rand(g, M, N, dtype=dtype, pad=pad) if residual else None
    y, z = _empty(M, N, dtype, pad=pad), _empty(M, N, dtype, pad=pad) if pre else None
    seed, offset = 77, 2**33 + 5
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    cuda_lib.dlrm_linear_fwd(x, w, b, r, y, pre=z, act=ref.ACT[name], p=p, rng=_rng(seed, offset),
                             workspace=_ws(cuda_lib.dlrm_linear_fwd_workspace_size(x, w)), status=status)
    kept, scale = ref.keep_scale(seed, offset, M, N, p) if p else (None, 1.0)
    wy, wz, ey, ez = ref.linear_fwd(_d(x), _d(w), _d(b), _d(r), name, kept, scale)
    ref.assert_close(y, wy, ey, dtype, "y")
    if pre:
        ref.assert_close(z, wz, ez, dtype, "pre")
        assert _guard_ok(z)
    assert _guard_ok(y) and int(status.item()) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("name,p,pad", [("none", 0.0, 0), ("relu", 0.1, 0), ("gelu", 0.0, 8), ("silu", 0.3, 3)])
def test_linear_bwd(cuda_lib, dtype, M, N, K, name, p, pad):
    g = torch.Generator().manual_seed(M + 31 * N + 977 * K + 1)
    x = _rand(g, M, K, dtype=dtype, pad=pad)
    w = _rand(g, N, K, std=K**-0.5, dtype=dtype, pad=pad)
    dy = _rand(g, M, N, std=0.1, dtype=dtype, pad=pad)
    z = _rand(g, M, N, dtype=dtype, pad=pad) if name != "none" else None
    dx, dw = _empty(M, K, dtype, pad=pad), _empty(N, K, dtype, pad=pad)
    db = torch.empty(N, device=dev())
    seed, offset = 78, 2**34 + 6
    code = ref.ACT[name]
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    ws = _ws(cuda_lib.dlrm_linear_bwd_workspace_size(dy, x, w, act=code, p=p))
    cuda_lib.dlrm_linear_bwd(dy, x, w, z, dx, dw, db, act=code, p=p, rng=_rng(seed, offset), workspace=ws,
                             status=status)
    kept, scale = ref.keep_scale(seed, offset, M, N, p) if p else (None, 1.0)
    want = ref.linear_bwd(_d(dy), _d(x), _d(w), _d(z), name, ref.U[dtype], kept, scale)
    ref.assert_close(dx, *want["dx"], dtype, "dx")
    ref.assert_close(dw, *want["dw"], dtype, "dw")
    ref.assert_close(db, *want["db"], "f32", "db")
    assert _guard_ok(dx) and _guard_ok(dw) and int(status.item()) == 0
    # each gradient alone has the same bits
    for only in range(3):
        o = [torch.empty_like(t) if i == only else None for i, t in enumerate((dx, dw, db))]
        cuda_lib.dlrm_linear_bwd(dy, x, w, z, *o, act=code, p=p, rng=_rng(seed, offset), workspace=ws)
        assert torch.equal(o[only], (dx, dw, db)[only])


@pytest.mark.parametrize("name", ["relu", "gelu", "silu"])
def test_linear_gradient_against_differences(cuda_lib, name):
    """Central differences of the forward itself, fp32: d/dh of sum(y * c) along random directions
    of x, w and b equals the backward's gradients.  h = 2^-6: the quotient's truncation error is below
    h^2 times the third derivative (under 1 for these functions at |z| of order 1, times the
    direction's cube), and its rounding error below 2^-16 of the sums' size."""
    M, N, K, p = 40, 24, 56, 0.25
    g = torch.Generator().manual_seed(3)
    x, w = _rand(g, M, K), _rand(g, N, K, std=K**-0.5)
    b, c = _rand(g, N), _rand(g, M, N, std=0.1)
    rng, code = _rng(4, 5), ref.ACT[name]

    def loss(x, w, b):
        y = torch.empty(M, N, device=dev())
        cuda_lib.dlrm_linear_fwd(x, w, b, None, y, act=code, p=p, rng=rng,
                                 workspace=_ws(cuda_lib.dlrm_linear_fwd_workspace_size(x, w)))
        return float((y.double() * c.double()).sum())

    z = torch.empty(M, N, device=dev())
    cuda_lib.dlrm_linear_fwd(x, w, b, None, torch.empty_like(z), pre=z, act=code, p=p, rng=rng,
                             workspace=_ws(cuda_lib.dlrm_linear_fwd_workspace_size(x, w)))
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    cuda_lib.dlrm_linear_bwd(c, x, w, z, dx, dw, db, act=code, p=p, rng=rng,
                             workspace=_ws(cuda_lib.dlrm_linear_bwd_workspace_size(c, x, w, act=code, p=p)))
    h = 2.0**-6
    for t, grad in ((0, dx), (1, dw), (2, db)):
        args = [x, w, b]
        v = _rand(g, *args[t].shape, std=0.2)
        hi, lo = [a.clone() for a in args], [a.clone() for a in args]
        hi[t] += h * v
        lo[t] -= h * v
        # a ReLU's kink: an element whose sign flips between the two ends is off by up to its slope;
        # the chance is h |v . w| a unit of density, so compare against the sum of absolute terms
        quotient = (loss(*hi) - loss(*lo)) / (2 * h)
        exact = float((grad.double() * v.double()).sum())
        size = float((grad.double().abs() * v.double().abs()).sum())
        assert abs(quotient - exact) <= (2.0**-6 if name == "relu" else 2.0**-9) * size, (name, t, quotient, exact, size)


def test_linear_dropout_is_dropout_of_the_layer(cuda_lib):
    """The layer's mask is dlrm_dropout_fwd's, whatever kernel runs (one row to many, odd widths)."""
    for M, N in ((1, 40), (5, 77), (200, 77), (400, 512)):
        g = torch.Generator().manual_seed(M)
        x, w = _rand(g, M, 64), _rand(g, N, 64, std=0.1)
        ws = _ws(cuda_lib.dlrm_linear_fwd_workspace_size(x, w))
        plain, both, after = (torch.empty(M, N, device=dev()) for _ in range(3))
        cuda_lib.dlrm_linear_fwd(x, w, None, None, plain, act=2, workspace=ws)
        cuda_lib.dlrm_linear_fwd(x, w, None, None, both, act=2, p=0.4, rng=_rng(1, 2), workspace=ws)
        cuda_lib.dlrm_dropout_fwd(plain, None, after, 0.4, _rng(1, 2))
        assert torch.equal(both, after)


def test_relu_gradient_from_its_output(cuda_lib):
    """For RELU without a residual the output serves as pre, dropout included."""
    M, N, K, p = 130, 72, 40, 0.3
    g = torch.Generator().manual_seed(8)
    x, w, dy = _rand(g, M, K, dtype="bf16"), _rand(g, N, K, std=0.2, dtype="bf16"), _rand(g, M, N, dtype="bf16")
    y, z = (torch.empty(M, N, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    rng = _rng(3, 3)
    cuda_lib.dlrm_linear_fwd(x, w, None, None, y, pre=z, act=1, p=p, rng=rng,
                             workspace=_ws(cuda_lib.dlrm_linear_fwd_workspace_size(x, w)))
    ws = _ws(cuda_lib.dlrm_linear_bwd_workspace_size(dy, x, w, act=1, p=p))
    outs = []
    for pre in (y, z):
        o = [torch.empty_like(x), torch.empty_like(w), torch.empty(N, device=dev())]
        cuda_lib.dlrm_linear_bwd(dy, x, w, pre, *o, act=1, p=p, rng=rng, workspace=ws)
        outs.append(o)
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [3, 200])
def test_linear_infinities_and_nan(cuda_lib, dtype, M):
    """One infinity or NaN in x reaches its own row alone, with the sign fp32 gives; one in w its own column."""
    N, K = 40, 72
    g = torch.Generator().manual_seed(1)
    x, w = _rand(g, M, K, dtype=dtype), _rand(g, N, K, std=0.1, dtype=dtype)
    x[0, 5], x[1, 70], w[3, 9] = INF, NAN, -INF
    y = torch.empty(M, N, dtype=ref.TYPES[dtype], device=dev())
    cuda_lib.dlrm_linear_fwd(x, w, None, None, y, workspace=_ws(cuda_lib.dlrm_linear_fwd_workspace_size(x, w)))
    want = _d(x) @ _d(w).t()
    out = _d(y)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(out[inf], want[inf]) and bool(torch.isfinite(out[torch.isfinite(want)]).all())
    assert int(torch.isfinite(want).sum()) == (M - 2) * (N - 1)


@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_no_rows(cuda_lib, dtype):
    N, K = 24, 40
    t = ref.TYPES[dtype]
    x, w, y = torch.empty(0, K, dtype=t, device=dev()), torch.ones(N, K, dtype=t, device=dev()), torch.empty(0, N, dtype=t, device=dev())
    assert cuda_lib.dlrm_linear_fwd_workspace_size(x, w) == 0
    cuda_lib.dlrm_linear_fwd(x, w, None, None, y)
    dw, db = _empty(N, K, dtype, pad=3), torch.ones(N, device=dev())
    cuda_lib.dlrm_linear_bwd(y, x, w, None, x, dw, db)
    assert bool((dw == 0).all()) and bool((db == 0).all()) and _guard_ok(dw)


def test_linear_reproducible_and_on_another_stream(cuda_lib):
    g = torch.Generator().manual_seed(2)
    M, N, K = 1000, 136, 264
    x, w, dy = _rand(g, M, K, dtype="f16"), _rand(g, N, K, std=0.1, dtype="f16"), _rand(g, M, N, dtype="f16")
    outs = []
    for stream in (None, None, torch.cuda.Stream()):
        torch.cuda.synchronize()
        o = [torch.empty_like(x), torch.empty_like(w), torch.empty(N, device=dev()), torch.empty_like(dy)]
        ws = _ws(cuda_lib.dlrm_linear_bwd_workspace_size(dy, x, w))
        wf = _ws(cuda_lib.dlrm_linear_fwd_workspace_size(x, w))
        cuda_lib.dlrm_linear_bwd(dy, x, w, None, *o[:3], workspace=ws, stream=stream)
        cuda_lib.dlrm_linear_fwd(x, w, None, None, o[3], workspace=wf, stream=stream)
        torch.cuda.synchronize()
        outs.append(o)
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], o))


def test_linear_in_a_graph_with_new_masks(cuda_lib):
    """A captured layer reads rng when it runs: advancing it between replays changes the mask."""
    g = torch.Generator().manual_seed(2)
    x, w = _rand(g, 64, 64, dtype="f16"), _rand(g, 64, 64, std=0.1, dtype="f16")
    y = torch.empty(64, 64, dtype=torch.float16, device=dev())
    rng = _rng(1, 0)
    ws = _ws(cuda_lib.dlrm_linear_fwd_workspace_size(x, w))
    cuda_lib.dlrm_linear_fwd(x, w, None, None, y, p=0.5, rng=rng, workspace=ws)
    first = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.dlrm_linear_fwd(x, w, None, None, y, p=0.5, rng=rng, workspace=ws)
        rng[1] += 1
    graph.replay()
    assert torch.equal(y, first)
    graph.replay()
    torch.cuda.synchronize()
    eager = torch.empty_like(y)
    cuda_lib.dlrm_linear_fwd(x, w, None, None, eager, p=0.5, rng=_rng(1, 1), workspace=ws)
    assert torch.equal(y, eager) and not torch.equal(y, first)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lead", [1, 2, 4])
def test_linear_misaligned_bases(cuda_lib, dtype, lead):
    """Operands that start off the 16-byte grid give the bits of aligned ones where the kernel is
    the same, and stay within the bounds everywhere."""
    for M, N, K in ((3, 40, 64), (200, 72, 64)):
        g = torch.Generator().manual_seed(lead)
        x, w = _rand(g, M, K, dtype=dtype, lead=lead, pad=8 - lead), _rand(g, N, K, std=0.1, dtype=dtype, lead=lead, pad=8 - lead)
        r = _rand(g, M, N, dtype=dtype, lead=lead, pad=8 - lead)
        y = torch.full((M, N + 8), 7.0, dtype=ref.TYPES[dtype], device=dev())[:, lead:lead + N]
        cuda_lib.dlrm_linear_fwd(x, w, None, r, y, act=2,
                                 workspace=_ws(cuda_lib.dlrm_linear_fwd_workspace_size(x, w)))
        wy, _, ey, _ = ref.linear_fwd(_d(x), _d(w), None, _d(r), "gelu")
        ref.assert_close(y, wy, ey, dtype)
        assert bool((y._base[:, :lead] == 7).all()) and bool((y._base[:, lead + N:] == 7).all())


def test_linear_many_rows_of_one_output(cuda_lib):
    """The logit layer of the training batch: 65,536 rows, 256 inputs, one output."""
    M, N, K = 65536, 1, 256
    g = torch.Generator().manual_seed(4)
    x, w, b = _rand(g, M, K, dtype="f16"), _rand(g, N, K, std=K**-0.5, dtype="f16"), _rand(g, N)
    y = torch.empty(M, N, dtype=torch.float16, device=dev())
    cuda_lib.dlrm_linear_fwd(x, w, b, None, y, workspace=_ws(cuda_lib.dlrm_linear_fwd_workspace_size(x, w)))
    wy, _, ey, _ = ref.linear_fwd(_d(x), _d(w), _d(b), None, "none")
    ref.assert_close(y, wy, ey, "f16")
    dy = _rand(g, M, N, dtype="f16")
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device=dev())
    cuda_lib.dlrm_linear_bwd(dy, x, w, None, dx, dw, db,
                             workspace=_ws(cuda_lib.dlrm_linear_bwd_workspace_size(dy, x, w)))
    want = ref.linear_bwd(_d(dy), _d(x), _d(w), None, "none", ref.U["f16"])
    for got, k, t in ((dx, "dx", "f16"), (dw, "dw", "f16"), (db, "db", "f32")):
        ref.assert_close(got, *want[k], t, k)


# ------------------------------------------------------------------------------------------- mixture of experts
def _moe_case(g, T, H, I, E, dtype, gated, pad=0):
    x = _rand(g, T, H, dtype=dtype, pad=pad)
    wr = _rand(g, E, H, std=H**-0.5, dtype=dtype).contiguous()
    w1 = _rand(g, E, I * (2 if gated else 1), H, std=H**-0.5, dtype=dtype).contiguous()
    w2 = _rand(g, E, H, I, std=I**-0.5, dtype=dtype).contiguous()
    return x, wr, w1, w2


def _run_moe(dl, x, wr, w1, w2, res, k, name, gated, pad=0):
    T, H = x.shape
    y = torch.full((T, H + pad), 7.0, dtype=x.dtype, device=dev())[:, :H]
    ids = torch.full((T, k), -1, dtype=torch.int32, device=dev())
    probs = torch.empty(T, k, device=dev())
    dl.dlrm_moe_fwd(x, wr, w1, w2, res, y, ids, probs, act=ref.ACT[name], gated=gated,
                    workspace=_ws(dl.dlrm_moe_fwd_workspace_size(x, wr, w1, w2, k)))
    return y, ids.cpu(), probs.cpu()


def _check_moe(x, wr, w1, w2, res, k, name, gated, dtype, y, ids, probs):
    want_ids, _ = ref.moe_route(_d(x) @ _d(wr).t(), k)
    # logits nearer than their rounding may change places: the choice must be as good
    logits = _d(x) @ _d(wr).t()
    near = (x.shape[1] + 8) * 2.0**-22 * (_d(x).abs() @ _d(wr).abs().t()).max()
    got = torch.gather(logits, 1, ids.long())
    assert bool(((got - torch.gather(logits, 1, want_ids)).abs() <= near).all())
    assert all(len(set(r)) == k for r in ids.tolist())
    wy, ey, wp, ep = ref.moe(_d(x), _d(wr), _d(w1), _d(w2), _d(res), ids.long(), name, gated,
                             ref.U[dtype] if dtype != "f32" else 0.0)
    ref.assert_close(probs, wp, ep, "f32", "probs")
    ref.assert_close(y, wy, ey, dtype, "y")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,I,E,k,name,gated,pad", [
    (1, 1, 1, 1, 1, "relu", False, 0), (1, 480, 1024, 8, 2, "silu", True, 0), (2, 40, 24, 3, 3, "gelu", False, 0),
    (5, 37, 19, 5, 2, "silu", True, 3), (7, 128, 64, 16, 4, "relu", False, 8), (8, 64, 72, 33, 8, "gelu", True, 0),
    (9, 256, 128, 2, 1, "silu", True, 0), (17, 96, 40, 7, 5, "none", True, 0), (33, 72, 48, 64, 6, "silu", True, 0),
    (64, 64, 32, 256, 8, "relu", False, 0), (64, 200, 136, 4, 4, "silu", True, 0), (48, 512, 256, 1, 1, "gelu", True, 0)])
def test_moe(cuda_lib, dtype, T, H, I, E, k, name, gated, pad):
    g = torch.Generator().manual_seed(T * 1000 + H)
    x, wr, w1, w2 = _moe_case(g, T, H, I, E, dtype, gated, pad)
    res = _rand(g, T, H, dtype=dtype, pad=pad) if T % 2 else None
    y, ids, probs = _run_moe(cuda_lib, x, wr, w1, w2, res, k, name, gated, pad)
    _check_moe(x, wr, w1, w2, res, k, name, gated, dtype, y, ids, probs)
    assert _guard_ok(y)


def test_moe_ties_and_wild_logits(cuda_lib):
    """Equal logits go to the lower index, -0 equals 0, NaN counts as largest; the ids are always
    different experts in range."""
    T, H, I, E, k = 4, 8, 8, 40, 8
    g = torch.Generator().manual_seed(6)
    _, _, w1, w2 = _moe_case(g, T, H, I, E, "f32", False)
    wr = torch.zeros(E, H, device=dev())
    x = torch.zeros(T, H, device=dev())
    x[0, 0] = 1.0                       # all logits 0 (some -0)
    wr[::3, 0] = -0.0
    x[1, 1], wr[7, 1], wr[35, 1] = 1.0, 2.0, 2.0   # 7 and 35 first, then zeros by index
    x[2, 2], wr[:, 2] = 1.0, -INF       # every logit -inf
    x[3, 3], wr[11, 3] = 1.0, NAN       # one NaN
    y, ids, probs = _run_moe(cuda_lib, x, wr, w1, w2, None, k, "relu", False)
    assert ids[0].tolist() == list(range(8))
    # rows 1 and 3 also meet the infinite column with a zero: 0 * inf is NaN everywhere
    for t in range(T):
        assert len(set(ids[t].tolist())) == k and all(0 <= e < E for e in ids[t].tolist())


def test_moe_ties_without_infinities(cuda_lib):
    T, H, I, E, k = 3, 8, 8, 40, 5
    g = torch.Generator().manual_seed(6)
    _, _, w1, w2 = _moe_case(g, T, H, I, E, "bf16", False)
    wr, x = torch.zeros(E, H, dtype=torch.bfloat16, device=dev()), torch.zeros(T, H, dtype=torch.bfloat16, device=dev())
    x[1, 1], wr[7, 1], wr[35, 1] = 1.0, 2.0, 2.0
    x[2, 2], wr[39, 2], wr[0, 2] = 1.0, 1.0, -1.0
    _, ids, probs = _run_moe(cuda_lib, x, wr, w1, w2, None, k, "relu", False)
    assert ids.tolist() == [[0, 1, 2, 3, 4], [7, 35, 0, 1, 2], [39, 1, 2, 3, 4]]
    assert torch.allclose(probs[0], torch.full((5,), 0.2), atol=1e-6)


def test_moe_nan_logit_is_chosen_first(cuda_lib):
    T, H, I, E, k = 1, 8, 8, 10, 3
    g = torch.Generator().manual_seed(6)
    _, _, w1, w2 = _moe_case(g, T, H, I, E, "f32", False)
    x, wr = torch.ones(T, H, device=dev()), torch.zeros(E, H, device=dev())
    wr[4, 0], wr[6, 0] = NAN, 1.0
    _, ids, _ = _run_moe(cuda_lib, x, wr, w1, w2, None, k, "relu", False)
    assert ids.tolist() == [[4, 6, 0]]


def test_moe_unchosen_experts_are_not_read_into_the_result(cuda_lib):
    """NaN weights of experts that no token chose leave the output as it was."""
    T, H, I, E, k = 3, 64, 32, 12, 2
    g = torch.Generator().manual_seed(9)
    x, wr, w1, w2 = _moe_case(g, T, H, I, E, "f16", True)
    y, ids, _ = _run_moe(cuda_lib, x, wr, w1, w2, None, k, "silu", True)
    for e in range(E):
        if not bool((ids == e).any()):
            w1[e], w2[e] = NAN, NAN
    y2, ids2, _ = _run_moe(cuda_lib, x, wr, w1, w2, None, k, "silu", True)
    assert torch.equal(y, y2) and torch.equal(ids, ids2)
    # nor does an expert reach a token that did not choose it
    e = int(ids[0, 0])
    w1[e, 0, 0], w2[e, 1, 1] = INF, NAN
    y3, _, _ = _run_moe(cuda_lib, x, wr, w1, w2, None, k, "silu", True)
    for t in range(T):
        if e not in ids[t].tolist():
            assert torch.equal(y3[t], y[t])
    assert bool(torch.isnan(y3[0]).any())


def test_moe_reproducible(cuda_lib):
    g = torch.Generator().manual_seed(10)
    x, wr, w1, w2 = _moe_case(g, 40, 256, 128, 24, "bf16", True)
    a = _run_moe(cuda_lib, x, wr, w1, w2, None, 4, "silu", True)
    for _ in range(3):
        b = _run_moe(cuda_lib, x, wr, w1, w2, None, 4, "silu", True)
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_moe_no_tokens(cuda_lib):
    x, wr = torch.empty(0, 16, device=dev()), torch.ones(4, 16, device=dev())
    w1, w2 = torch.ones(4, 8, 16, device=dev()), torch.ones(4, 16, 8, device=dev())
    cuda_lib.dlrm_moe_fwd(x, wr, w1, w2, None, torch.empty(0, 16, device=dev()),
                          torch.empty(0, 2, dtype=torch.int32, device=dev()), torch.empty(0, 2, device=dev()), gated=False)
