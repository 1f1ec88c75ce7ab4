"""The residual blocks' operators as programs use them: a block of experts forward and backward against
autograd in 64 bits, captured graphs, other streams, two calls at once, matrices past 2^32 bytes."""

import os
import sys

import pytest
import torch

import block_ref as ref
import dense_ref as dref
from gpu_util import dev

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_mixture
    finally:
        sys.path.pop(0)
    return train_mixture


def _ws(n):
    return torch.empty(n, dtype=torch.uint8, device=dev()) if n else None


def _block_in_64_bits(block, x, ids):
    """(r, next h, {name: leaf}) of the block on x, the experts' choice given."""
    leaf = {n: v.double().cpu().requires_grad_() for n, v in block.p.items()}
    leaf["x"] = x.double().cpu().requires_grad_()

    def rms(v):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)

    h = rms(leaf["x"])
    probs = torch.softmax(torch.gather(h @ leaf["router"].t(), 1, ids), 1)
    m = torch.zeros_like(h)
    for e in range(leaf["w1"].shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        z = h[t] @ leaf["w1"][e].t() + leaf["b1"][e]
        m = m.index_add(0, t, probs[t, j][:, None] * (torch.nn.functional.gelu(z) @ leaf["w2"][e].t()))
    r = leaf["x"] + leaf["scale"] * torch.sigmoid(h @ leaf["gate"].t()) * rms(m) * leaf["w_post"]
    return r, rms(r) * leaf["w_next"], leaf


@pytest.mark.parametrize("T,H,hidden,E,k", [(65, 72, 40, 5, 2), (3, 48, 24, 6, 3), (200, 64, 33, 4, 1)])
def test_block_of_experts_against_autograd(cuda_lib, example, T, H, hidden, E, k):
    """Every gradient of the block, fp32.  The longest chain sums H, hidden, k, H and T terms one after
    another, each to (L + 8) 2^-23 of its terms' sizes, which cancel to a tenth at most: in all within
    (3 H + 2 hidden + T + 50) 2^-23 * 10 of the gradient's largest value."""
    block = example.MixtureBlock(H, hidden, E, k, seed=T)
    g = torch.Generator().manual_seed(T)
    block.p["scale"].copy_(torch.rand(H, generator=g) + 0.5)
    x, cr, ch = (torch.randn(T, H, generator=g).to(dev()) for _ in range(3))
    h, stats = example.first_norm(x)
    r, nh = block.forward(x, h)
    gx, gh = block.backward(cr, ch)
    gx = example.first_norm_grad(x, stats, gx, gh)
    rr, rh, leaf = _block_in_64_bits(block, x, block.kept["ids"].cpu().long())
    ((rr * cr.double().cpu()).sum() + (rh * ch.double().cpu()).sum()).backward()
    tol = (3 * H + 2 * hidden + T + 50) * 2.0**-23 * 10
    for name, got, want in [("r", r, rr), ("h", nh, rh), ("x", gx, leaf["x"].grad)] + \
            [(n, block.g[n], leaf[n].grad) for n in block.p]:
        got, want = got.double().cpu(), want.detach()
        assert float((got - want).abs().max()) <= tol * float(want.abs().max()), name


def test_block_with_activations_in_8_bits(cuda_lib, example):
    """The forward and the gradients of what does not pass an expert's kept values are the same; w2's
    gradient is off by its inputs' rounding: half a step of four bits, 2^-4 of each, or for the least
    values 2^-17 of their block's largest."""
    T, H, hidden, E, k = 300, 64, 96, 4, 2
    full, small = (example.MixtureBlock(H, hidden, E, k, bits8=b, seed=1) for b in (False, True))
    g = torch.Generator().manual_seed(2)
    x, cr, ch = (torch.randn(T, H, generator=g).to(dev()) for _ in range(3))
    h, _ = example.first_norm(x)
    outs = [b.forward(x, h) for b in (full, small)]
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    for b in (full, small):
        b.backward(cr, ch)
    for n in ("w_post", "scale", "w_next", "gate", "router"):
        assert torch.equal(full.g[n], small.g[n]), n
    s = full.kept
    at = s["at"]
    gm = torch.empty_like(x)
    cuda_lib.dlrm_block_norm_bwd(cr, ch, s["m"], s["gate"], s["r"], s["stats"], full.p["w_post"], None, full.p["scale"],
                                 full.p["w_next"], gm, None, None, *[None] * 5, **example.NORM)
    gys = torch.zeros_like(s["ys"])
    cuda_lib.dlrm_combine_bwd(gm, None, s["slots"], s["probs"], gys, None)
    a = s["a"].double()
    off = torch.maximum(a.abs() * 2.0**-4, a.view(-1, hidden // 32, 32).abs().amax(2).repeat_interleave(32, 1) * 2.0**-17)
    for e in range(E):
        rows = slice(at[e], at[e + 1])
        size = gys[rows].double().abs().t()
        bound = size @ off[rows] + (T + 8) * 2.0**-22 * (size @ a[rows].abs())
        assert bool(((full.g["w2"][e].double() - small.g["w2"][e].double()).abs() <= bound + 1e-12).all())


def test_example_runs(cuda_lib, example):
    for bits8 in (False, True):
        losses = example.train(3, tokens=64, width=64, bits8=bits8)
        assert len(losses) == 3 and all(v == v and v < float("inf") for v in losses)
        assert example.train(3, tokens=64, width=64, bits8=bits8) == losses


class Step:
    """One pass through every operator on buffers of its own."""

    def __init__(self, dl, dtype, T=700, H=200, E=33, k=3, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.dl, t = dl, dref.TYPES[dtype]
        d = dict(device=dev())
        self.x, self.y, self.gate, self.gr, self.gh = (torch.randn(T, H, generator=g).to(t).to(dev()) for _ in range(5))
        self.logits = torch.randn(T, E, generator=g).to(t).to(dev())
        self.w = torch.randn(H, H, generator=g).to(t).to(dev())
        self.v = [torch.rand(H, generator=g).to(dev()) for _ in range(5)]
        self.E = E
        m = lambda r=T, c=H, dtype=t: torch.zeros(r, c, dtype=dtype, **d)
        i32, u8, f32 = torch.int32, torch.uint8, torch.float32
        self.o = dict(r=m(), h=m(), stats=m(T, 4, f32), ids=m(T, k, i32), probs=m(T, k, f32), off=torch.zeros(E + 1, dtype=i32, **d),
                      slots=m(T, k, i32), order=torch.zeros(T * k, dtype=i32, **d), xs=m(T * k), c=m(), gxs=m(T * k), gp=m(T, k, f32),
                      gx=m(), gl=m(T, E), q=m(T, H, u8), e=m(T, (H + 31) // 32, u8), back=m(), ga=m(), gb=m(), gres=m(),
                      gv=m(5, H, f32), dx=m(), dw=m(H, H), db=torch.zeros(H, **d))
        o = self.o
        self.ws = [_ws(dl.dlrm_expert_sort_workspace_size(o["ids"], E)), _ws(dl.dlrm_block_norm_bwd_workspace_size(self.x)),
                   _ws(dl.dlrm_linear_bwd8_workspace_size(self.gr, o["q"], self.w, act=2))]

    def run(self, stream=None):
        dl, o, v, s = self.dl, self.o, self.v, dict(stream=stream)
        n = dict(norm=1, gate_act=2, stream=stream)
        dl.dlrm_block_norm_fwd(self.y, self.gate, self.x, *v, o["r"], o["h"], o["stats"], **n)
        dl.dlrm_route_fwd(self.logits, o["ids"], o["probs"], **s)
        dl.dlrm_expert_sort(o["ids"], self.E, o["off"], o["slots"], o["order"], workspace=self.ws[0], **s)
        dl.dlrm_dispatch_fwd(o["h"], o["slots"], o["xs"], **s)
        dl.dlrm_combine_fwd(o["xs"], o["slots"], o["probs"], o["r"], o["c"], **s)
        dl.dlrm_pack8(o["c"], o["q"], o["e"], **s)
        dl.dlrm_unpack8(o["q"], o["e"], o["back"], **s)
        dl.dlrm_linear_bwd8(self.gr, o["q"], o["e"], self.w, o["q"], o["e"], o["dx"], o["dw"], o["db"], act=2, workspace=self.ws[2], **s)
        dl.dlrm_combine_bwd(o["dx"], o["xs"], o["slots"], o["probs"], o["gxs"], o["gp"], **s)
        dl.dlrm_dispatch_bwd(o["gxs"], o["slots"], o["gx"], **s)
        dl.dlrm_route_bwd(o["gp"], o["ids"], o["probs"], o["gl"], **s)
        dl.dlrm_block_norm_bwd(self.gr, o["gx"], self.y, self.gate, o["r"], o["stats"], *v[:4], o["ga"], o["gb"], o["gres"],
                               *o["gv"].unbind(0), workspace=self.ws[1], **n)

    def outputs(self):
        return {n: t.clone() for n, t in self.o.items()}


def _same(a, b):
    return [n for n in a if not torch.equal(a[n].nan_to_num(7.0) if a[n].is_floating_point() else a[n],
                                            b[n].nan_to_num(7.0) if b[n].is_floating_point() else b[n])] == []


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H", [200, 77])
def test_captured_on_another_stream_and_beside_another(cuda_lib, dtype, H):
    a = Step(cuda_lib, dtype, H=H)
    first, second = (a.x.clone(), a.logits.clone()), (a.x.flip(0).contiguous(), a.logits.flip(0).contiguous())
    want = []
    for x, l in (first, second):
        a.x.copy_(x)
        a.logits.copy_(l)
        a.run()
        want.append(a.outputs())
    assert not torch.equal(want[0]["ids"], want[1]["ids"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    for (x, l), w in ((first, want[0]), (second, want[1]), (first, want[0])):
        a.x.copy_(x)
        a.logits.copy_(l)
        for t in a.o.values():
            t.zero_()
        graph.replay()
        assert _same(a.outputs(), w)
    b = Step(cuda_lib, dtype, H=H)
    b.x.copy_(second[0])
    b.logits.copy_(second[1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):      # both at once, each with its own workspaces
        a.run(streams[0])
        b.run(streams[1])
    torch.cuda.synchronize()
    assert _same(a.outputs(), want[0]) and _same(b.outputs(), want[1])


def test_rows_past_2_32_bytes_apart(cuda_lib):
    """Rows 2^31 + 64 elements apart in one 8-byte-a-row-sized buffer: every offset passes 32 bits."""
    dl, far, N = cuda_lib, 2**31 + 64, 96
    base = torch.empty(2 * far + 4 * N, dtype=torch.bfloat16, device=dev())
    view = lambda at: base.as_strided((3, N), (far, 1), at)
    x, y = view(0), view(N)
    g = torch.Generator().manual_seed(0)
    near = torch.randn(3, N, generator=g).bfloat16().to(dev())
    x.copy_(near)
    h, hn = view(2 * N), torch.empty_like(near)
    dl.dlrm_block_norm_fwd(x, None, x, None, None, None, None, None, y, h)
    rn = torch.empty_like(near)
    dl.dlrm_block_norm_fwd(near, None, near, None, None, None, None, None, rn, hn)
    assert torch.equal(y, rn) and torch.equal(h, hn)
    slots = torch.tensor([[2], [0], [1]], dtype=torch.int32, device=dev())
    dl.dlrm_dispatch_fwd(x, slots, h)
    assert torch.equal(h[[2, 0, 1]], near)
    dl.dlrm_dispatch_bwd(h, slots, y)
    assert torch.equal(y, near)
    q, e, back = base.view(torch.uint8).as_strided((3, N), (2 * far, 1), 6 * N), torch.empty(3, 3, dtype=torch.uint8, device=dev()), view(2 * N)
    dl.dlrm_pack8(x, q, e)
    rq, re = ref.pack8(near.double().cpu())
    assert torch.equal(q.cpu().long(), rq) and torch.equal(e.cpu().long(), re)
    dl.dlrm_unpack8(q, e, back)
    assert torch.equal(back.double().cpu(), ref.unpack8(rq, re, 3.3895313892515355e38))


def test_a_matrix_of_more_than_2_31_elements(cuda_lib):
    """Rows of 2^17 columns to 2^14 + 3 places: the last elements' numbers pass 2^31."""
    T, H = (2**14 + 3) // 2, 2**17 + 8
    x = torch.empty(T, H, dtype=torch.float16, device=dev())
    x.copy_((torch.arange(T, device=dev())[:, None] % 1024).half().expand(T, H))
    x[:, -1] = 7.0
    slots = torch.stack((torch.arange(T, device=dev()), 2 * T - 1 - torch.arange(T, device=dev())), 1).int().contiguous()
    xs = torch.empty(2 * T, H, dtype=torch.float16, device=dev())
    assert xs.numel() > 2**31
    cuda_lib.dlrm_dispatch_fwd(x, slots, xs)
    assert torch.equal(xs[:T], x) and torch.equal(xs[T:], x.flip(0))
    cuda_lib.dlrm_dispatch_bwd(xs, slots, x)
    assert bool((x[:, 0] == 2 * (torch.arange(T, device=dev()) % 1024)).all()) and bool((x[:, -1] == 14.0).all())
    q, e = torch.empty(2 * T, H, dtype=torch.uint8, device=dev()), torch.empty(2 * T, (H + 31) // 32, dtype=torch.uint8, device=dev())
    cuda_lib.dlrm_pack8(xs, q, e)
    cuda_lib.dlrm_unpack8(q, e, xs)
    assert bool((xs[:, -1] == 7.0).all()) and torch.equal(xs[:16, 0], torch.arange(16, device=dev()).half())
