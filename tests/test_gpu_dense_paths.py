"""The dense network's larger tiles and its failure detection, and the example that runs its
operators together with the lookup and the interaction."""

import os
import sys

import pytest
import torch

import dense_ref as ref
from gpu_util import dev

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _rand(g, *shape, std=1.0, dtype="f32"):
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * std).to(ref.TYPES[dtype]).to(dev())


def _ws(n):
    return torch.empty(n, dtype=torch.uint8, device=dev()) if n else None


def _rng(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device=dev())


def _gpu64(bound_of, *args):
    """dense_ref on the GPU's own 64-bit arithmetic (these products are too large for the host)."""
    return bound_of(*[a.double() if isinstance(a, torch.Tensor) and a.is_floating_point() else a for a in args])


# block pairs of 256 x 256 and 256 x 128, single blocks, split K, ragged last tiles, several tiles a block; few outputs
LARGE = [(8192, 1024, 480, "f16"), (40000, 264, 72, "bf16"), (2048, 512, 4096, "f16"), (300, 1032, 2056, "bf16"),
         (5003, 515, 367, "f32"), (1024, 2048, 264, "f32"), (20000, 40, 1024, "bf16"), (70000, 8, 24, "f16"),
         (40000, 13, 600, "f32"), (40000, 1, 256, "f16"), (2000, 5, 1304, "bf16"), (2000, 16, 1300, "f32")]


@pytest.mark.parametrize("M,N,K,dtype", LARGE)
@pytest.mark.parametrize("name,p,residual", [("relu", 0.1, False), ("gelu", 0.0, True)])
def test_large_forward(cuda_lib, M, N, K, dtype, name, p, residual):
    g = torch.Generator().manual_seed(M)
    x, w, b = _rand(g, M, K, dtype=dtype), _rand(g, N, K, std=K**-0.5, dtype=dtype), _rand(g, N)
    r = _rand(g, M, N, dtype=dtype) if residual else None
    y, z = (torch.empty(M, N, dtype=ref.TYPES[dtype], device=dev()) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    cuda_lib.dlrm_linear_fwd(x, w, b, r, y, pre=z, act=ref.ACT[name], p=p, rng=_rng(3, 4), status=status,
                             workspace=_ws(cuda_lib.dlrm_linear_fwd_workspace_size(x, w)))
    kept, scale = ref.keep_scale(3, 4, M, N, p) if p else (None, 1.0)
    kept = kept.to(dev()) if kept is not None else None
    wy, wz, ey, ez = _gpu64(ref.linear_fwd, x, w, b, r, name, kept, scale)
    ref.assert_close(y, wy, ey, dtype, "y")
    ref.assert_close(z, wz, ez, dtype, "pre")
    assert int(status.item()) == 0


@pytest.mark.parametrize("M,N,K,dtype", LARGE)
@pytest.mark.parametrize("name,p", [("relu", 0.1), ("silu", 0.0)])
def test_large_backward(cuda_lib, M, N, K, dtype, name, p):
    g = torch.Generator().manual_seed(M + 1)
    x, w, dy = _rand(g, M, K, dtype=dtype), _rand(g, N, K, std=K**-0.5, dtype=dtype), _rand(g, M, N, std=0.1, dtype=dtype)
    z = _rand(g, M, N, dtype=dtype)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device=dev())
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    code = ref.ACT[name]
    cuda_lib.dlrm_linear_bwd(dy, x, w, z, dx, dw, db, act=code, p=p, rng=_rng(5, 6), status=status,
                             workspace=_ws(cuda_lib.dlrm_linear_bwd_workspace_size(dy, x, w, act=code, p=p)))
    kept, scale = ref.keep_scale(5, 6, M, N, p) if p else (None, 1.0)
    kept = kept.to(dev()) if kept is not None else None
    want = _gpu64(ref.linear_bwd, dy, x, w, z, name, ref.U[dtype], kept, scale)
    ref.assert_close(dx, *want["dx"], dtype, "dx")
    ref.assert_close(dw, *want["dw"], dtype, "dw")
    ref.assert_close(db, *want["db"], "f32", "db")
    assert int(status.item()) == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 8, 9, 13, 16])
@pytest.mark.parametrize("M,K,pad", [(1, 1, 0), (5, 8, 0), (40, 520, 0), (31, 1027, 3), (513, 64, 8), (9001, 250, 0),
                                     (66000, 16, 0)])
def test_few_outputs_backward(cuda_lib, dtype, N, M, K, pad):
    """One row chunk and many, rows on and off the 16-byte grid, several column blocks, every count of
    outputs a kernel is made for and those between; each gradient alone has the same bits."""
    g = torch.Generator().manual_seed(M + N)
    x, w = (_rand(g, r, K + pad, dtype=dtype)[:, :K] for r in (M, N))
    dy, z = _rand(g, M, N + pad, std=0.1, dtype=dtype)[:, :N], _rand(g, M, N, dtype=dtype)
    dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros(N, device=dev())
    code, p = ref.ACT["gelu"], 0.2
    ws = _ws(cuda_lib.dlrm_linear_bwd_workspace_size(dy, x, w, act=code, p=p))
    cuda_lib.dlrm_linear_bwd(dy, x, w, z, dx, dw, db, act=code, p=p, rng=_rng(8, 9), workspace=ws)
    kept, scale = ref.keep_scale(8, 9, M, N, p)
    want = _gpu64(ref.linear_bwd, dy, x, w, z, "gelu", ref.U[dtype], kept.to(dev()), scale)
    ref.assert_close(dx, *want["dx"], dtype, "dx")
    ref.assert_close(dw, *want["dw"], dtype, "dw")
    ref.assert_close(db, *want["db"], "f32", "db")
    for only in range(3):
        o = [torch.empty_like(t) if i == only else None for i, t in enumerate((dx, dw, db))]
        cuda_lib.dlrm_linear_bwd(dy, x, w, z, *o, act=code, p=p, rng=_rng(8, 9), workspace=ws)
        assert torch.equal(o[only], (dx, dw, db)[only])


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("M,N,K,dtype", [(256, 512, 1024, "bf16"), (3000, 515, 130, "f32"), (5000, 64, 2056, "f16"),
                                         (200, 100, 13, "f16"), (3000, 8, 130, "bf16")])
def test_gradients_back_to_back(cuda_lib, M, N, K, dtype, graph):
    """A call's kernels overlap one another, never those of the call before or after: gradients in one
    workspace, each fed by the last one's dX, have the bits of calls with a synchronize between."""
    g = torch.Generator().manual_seed(K)
    w, z, dy = _rand(g, N, K, std=K**-0.5, dtype=dtype), _rand(g, M, N, dtype=dtype), _rand(g, M, N, dtype=dtype)
    x0 = _rand(g, M, K, dtype=dtype)
    ws = _ws(cuda_lib.dlrm_linear_bwd_workspace_size(dy, x0, w, act=3, p=0.1))
    steps = 8
    dx = [torch.zeros_like(x0) for _ in range(steps)]
    dw, db = [torch.zeros_like(w) for _ in range(steps)], [torch.zeros(N, device=dev()) for _ in range(steps)]
    rng = _rng(2, 3)

    def run(sync):
        for i in range(steps):
            cuda_lib.dlrm_linear_bwd(dy, dx[i - 1] if i else x0, w, z, dx[i], dw[i], db[i], act=3, p=0.1, rng=rng, workspace=ws)
            dy.mul_(-1)
            if sync:
                torch.cuda.synchronize()

    run(True)
    want = [t.clone() for t in dx + dw + db]
    for t in dx + dw + db:
        t.zero_()
    if graph:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(False)
        graph.replay()
    else:
        run(False)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(dx + dw + db, want))


@pytest.fixture
def wait_limit(cuda_lib):
    """Restores the wait limit whatever the test does."""
    yield cuda_lib.dlrm_set_wait_limit
    cuda_lib.dlrm_set_wait_limit(-1)


@pytest.mark.parametrize("M,N,K,dtype", [(8192, 1024, 480, "f16"), (300, 200, 264, "bf16"), (1024, 96, 1024, "f32")])
def test_linear_reports_a_wait_that_gives_up(cuda_lib, wait_limit, M, N, K, dtype):
    """With a limit of 0 cycles the first wait that is not already over gives up: the call sets
    DLRM_STATUS_TIMEOUT and returns, and the next call with the default limit is right."""
    g = torch.Generator().manual_seed(1)
    x, w, r = _rand(g, M, K, dtype=dtype), _rand(g, N, K, std=K**-0.5, dtype=dtype), _rand(g, M, N, dtype=dtype)
    ws = _ws(cuda_lib.dlrm_linear_fwd_workspace_size(x, w))
    y, good = (torch.empty(M, N, dtype=ref.TYPES[dtype], device=dev()) for _ in range(2))
    cuda_lib.dlrm_linear_fwd(x, w, None, r, good, workspace=ws)
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    wait_limit(0)
    cuda_lib.dlrm_linear_fwd(x, w, None, r, y, workspace=ws, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == cuda_lib.DLRM_STATUS_TIMEOUT
    wait_limit(-1)
    status.zero_()
    cuda_lib.dlrm_linear_fwd(x, w, None, r, y, workspace=ws, status=status)
    assert torch.equal(y, good) and int(status.item()) == 0


def test_moe_reports_a_wait_that_gives_up(cuda_lib, wait_limit):
    """200 MB of weights: HBM brings them more slowly than the warps take them, so some wait is not over
    when it begins (the weights of a small mixture come out of L2 before they are waited for)."""
    T, H, I, E, k = 16, 2048, 512, 32, 8
    g = torch.Generator(device=dev())
    g.manual_seed(2)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=dev(), dtype=torch.float16).mul_(shape[-1]**-0.5)

    x, wr, w1, w2 = rand(T, H).mul_(H**0.5), rand(E, H), rand(E, 2 * I, H), rand(E, H, I)
    ws = _ws(cuda_lib.dlrm_moe_fwd_workspace_size(x, wr, w1, w2, k))
    ids, probs = torch.empty(T, k, dtype=torch.int32, device=dev()), torch.empty(T, k, device=dev())
    y, good = torch.empty_like(x), torch.empty_like(x)
    cuda_lib.dlrm_moe_fwd(x, wr, w1, w2, None, good, ids, probs, workspace=ws)
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    wait_limit(0)
    cuda_lib.dlrm_moe_fwd(x, wr, w1, w2, None, y, ids, probs, workspace=ws, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == cuda_lib.DLRM_STATUS_TIMEOUT
    wait_limit(-1)
    status.zero_()
    cuda_lib.dlrm_moe_fwd(x, wr, w1, w2, None, y, ids, probs, workspace=ws, status=status)
    assert torch.equal(y, good) and int(status.item()) == 0


def test_moe_wide(cuda_lib):
    """Rows longer than a stage, more units than warps, an expert with more tokens than are multiplied at once."""
    for T, H, I, E, k, dtype in ((50, 1024, 512, 3, 2, "bf16"), (40, 1032, 1000, 12, 3, "f32"), (64, 2048, 64, 1, 1, "f16")):
        g = torch.Generator().manual_seed(T)
        x, wr = _rand(g, T, H, dtype=dtype), _rand(g, E, H, std=H**-0.5, dtype=dtype)
        w1, w2 = _rand(g, E, 2 * I, H, std=H**-0.5, dtype=dtype), _rand(g, E, H, I, std=I**-0.5, dtype=dtype)
        y, probs = torch.empty_like(x), torch.empty(T, k, device=dev())
        ids = torch.empty(T, k, dtype=torch.int32, device=dev())
        cuda_lib.dlrm_moe_fwd(x, wr, w1, w2, None, y, ids, probs,
                              workspace=_ws(cuda_lib.dlrm_moe_fwd_workspace_size(x, wr, w1, w2, k)))
        d = [t.double().cpu() for t in (x, wr, w1, w2)]
        wy, ey, wp, ep = ref.moe(*d, None, ids.cpu().long(), "silu", True, ref.U[dtype] if dtype != "f32" else 0.0)
        ref.assert_close(probs, wp, ep, "f32", "probs")
        ref.assert_close(y, wy, ey, dtype, "y")


def test_example_trains_and_scores(cuda_lib):
    """examples/train_and_score.py: the loss of 40 steps falls by a third, twice the same; scoring returns
    finite logits through distinct experts."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_and_score as example
    finally:
        sys.path.pop(0)
    model, losses = example.train(40)
    assert losses[-1] < losses[0] * 2 / 3, losses
    assert example.train(40)[1] == losses
    logit, ids, probs = example.score(model)
    assert bool(torch.isfinite(logit).all()) and all(len(set(r)) == 2 for r in ids.tolist())
    assert torch.allclose(probs.sum(1), torch.ones(4, device=dev()), atol=1e-6)
