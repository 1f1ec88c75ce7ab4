"""The dense network as programs use it: operands that start anywhere, captured graphs, other streams;
and the mixture's choice where logits are not numbers."""

import pytest
import torch

import dense_ref as ref
from gpu_util import dev

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def _rand(g, *shape, std=1.0, dtype="f32"):
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * std).to(ref.TYPES[dtype]).to(dev())


def _ws(n):
    return torch.empty(n, dtype=torch.uint8, device=dev()) if n else None


def _inside(M, N, dtype, lead, values=None):
    """An M x N matrix that starts `lead` elements into rows of N + 8, with 7.0 around it."""
    t = torch.full((M, N + 8), 7.0, dtype=ref.TYPES[dtype], device=dev())[:, lead:lead + N]
    if values is not None:
        t.copy_(values)
    return t


def _untouched(t, lead):
    return bool((t._base[:, :lead] == 7).all()) and bool((t._base[:, lead + t.shape[1]:] == 7).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lead", [1, 2, 4])
@pytest.mark.parametrize("M,N,K", [(200, 72, 64), (3, 40, 64), (1500, 136, 264), (300, 8, 64), (300, 5, 67)])
@pytest.mark.parametrize("name,p", [("none", 0.0), ("relu", 0.2), ("gelu", 0.0)])
def test_gradient_of_misaligned_operands(cuda_lib, dtype, lead, M, N, K, name, p):
    g = torch.Generator().manual_seed(M + lead)
    x, w = _inside(M, K, dtype, lead, _rand(g, M, K)), _inside(N, K, dtype, lead, _rand(g, N, K, std=K**-0.5))
    dy, z = _inside(M, N, dtype, lead, _rand(g, M, N, std=0.1)), _inside(M, N, dtype, lead, _rand(g, M, N))
    dx, dw, db = _inside(M, K, dtype, lead), _inside(N, K, dtype, lead), torch.zeros(N + 1, device=dev())[1:]
    rng = torch.tensor([8, 9], device=dev())
    code = ref.ACT[name]
    cuda_lib.dlrm_linear_bwd(dy, x, w, z, dx, dw, db, act=code, p=p, rng=rng,
                             workspace=_ws(cuda_lib.dlrm_linear_bwd_workspace_size(dy, x, w, act=code, p=p)))
    kept, scale = ref.keep_scale(8, 9, M, N, p) if p else (None, 1.0)
    want = ref.linear_bwd(*[t.double().cpu() for t in (dy, x, w, z)], name, ref.U[dtype], kept, scale)
    ref.assert_close(dx, *want["dx"], dtype, "dx")
    ref.assert_close(dw, *want["dw"], dtype, "dw")
    ref.assert_close(db, *want["db"], "f32", "db")
    assert _untouched(dx, lead) and _untouched(dw, lead)


class Mixture:
    def __init__(self, dl, dtype, H, I, T=6, E=8, k=2, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.dl, self.k = dl, k
        self.x, self.wr = _rand(g, T, H, dtype=dtype), _rand(g, E, H, std=H**-0.5, dtype=dtype)
        self.w1, self.w2 = _rand(g, E, 2 * I, H, std=H**-0.5, dtype=dtype), _rand(g, E, H, I, std=I**-0.5, dtype=dtype)
        self.y = torch.zeros_like(self.x)
        self.ids, self.probs = torch.zeros(T, k, dtype=torch.int32, device=dev()), torch.zeros(T, k, device=dev())
        self.ws = _ws(dl.dlrm_moe_fwd_workspace_size(self.x, self.wr, self.w1, self.w2, k))

    def run(self, stream=None):
        self.dl.dlrm_moe_fwd(self.x, self.wr, self.w1, self.w2, self.x, self.y, self.ids, self.probs, workspace=self.ws,
                             stream=stream)
        return self

    def outputs(self):
        return [t.clone() for t in (self.y, self.ids, self.probs)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H,I", [(256, 128), (67, 35)])
def test_mixture_in_a_graph_and_on_another_stream(cuda_lib, dtype, H, I):
    """A captured mixture chooses anew at each replay; another stream gives the same bits."""
    m = Mixture(cuda_lib, dtype, H, I)
    a, b = m.x.clone(), m.x.flip(0).contiguous()
    want = []
    for x in (a, b):
        m.x.copy_(x)
        want.append(m.run().outputs())
    assert not torch.equal(want[0][1], want[1][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.run()
    for x, w in ((a, want[0]), (b, want[1]), (a, want[0])):
        m.x.copy_(x)
        graph.replay()
        assert all(torch.equal(s, t) for s, t in zip(m.outputs(), w))
    stream = torch.cuda.Stream()
    m.x.copy_(b)
    torch.cuda.synchronize()
    m.run(stream)
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(m.outputs(), want[1]))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_mixture_choice_where_logits_are_not_numbers(cuda_lib, dtype):
    """The largest first, a NaN above all, equal ones by lower index: every id is determined."""
    T, H, I, E, k = 5, 8, 8, 40, 8
    m = Mixture(cuda_lib, dtype, H, I, T, E, k)
    m.x.zero_()
    m.wr.zero_()
    m.wr[:, 2] = -INF                        # meets a 0 of every token but the third: 0 * inf is a NaN
    m.wr[11, 3] = NAN
    m.x[2, 2] = 1.0                          # -inf everywhere, NaN at 11
    assert m.run().ids.tolist() == [list(range(8))] * 2 + [[11] + list(range(7))] + [list(range(8))] * 2
    m.wr[:, 2], m.wr[11, 3] = 0.0, 0.0
    m.x.zero_()
    m.x[0, 0], m.wr[::3, 0] = 1.0, -0.0      # all 0, some of them -0
    m.x[1, 1], m.wr[7, 1], m.wr[35, 1] = 1.0, 2.0, 2.0
    m.x[2, 3], m.wr[4, 3], m.wr[9, 3] = 1.0, INF, -INF
    m.x[3, 4], m.wr[39, 4], m.wr[38, 4] = 1.0, 1.0, 1.0
    # an infinite weight makes the logits of tokens with a 0 there NaN: experts 4 and 9 come first for them
    got = m.run().ids.tolist()
    assert got[0] == [4, 9, 0, 1, 2, 3, 5, 6] and got[1] == [4, 9, 7, 35, 0, 1, 2, 3]
    assert got[2] == [4, 0, 1, 2, 3, 5, 6, 7] and got[3] == [4, 9, 38, 39, 0, 1, 2, 3] and got[4] == got[0]
