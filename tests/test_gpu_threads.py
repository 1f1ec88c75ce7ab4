"""Calls from threads that have made none before (no context is current there yet), alone and several
at once: every entry point that encodes tensor maps has the bits of the main thread's call."""

import threading

import pytest
import torch

import dense_ref as ref
from gpu_util import dev

pytestmark = pytest.mark.gpu


def _rand(g, *shape, std=1.0, dtype="f32"):
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * std).to(ref.TYPES[dtype]).to(dev())


def _ws(n):
    return torch.empty(n, dtype=torch.uint8, device=dev()) if n else None


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


def _in_new_thread(fn):
    errors = []

    def run():
        try:
            fn()
        except Exception as e:      # noqa: BLE001
            errors.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert not errors, errors


def _cases(dl):
    """{name: (call(stream), outputs)}"""
    g = torch.Generator().manual_seed(1)
    F, D, B, P = 26, 128, 300, 480
    dense, pooled = _rand(g, B, D, dtype="f16"), _rand(g, B, F, D, std=0.1, dtype="f16")
    out, gd, gp = torch.zeros(B, P, device=dev()).half(), torch.zeros_like(dense), torch.zeros_like(pooled)
    go = _rand(g, B, P, dtype="f16")
    m = Mixture(dl, "f16", 256, 128)
    x, w = _rand(g, 300, 64, dtype="f16"), _rand(g, 96, 64, std=0.1, dtype="f16")
    dy = _rand(g, 300, 96, dtype="f16")
    y, dx, dw, db = torch.zeros(300, 96, device=dev()).half(), torch.zeros_like(x), torch.zeros_like(w), torch.zeros(96, device=dev())
    wf, wb = _ws(dl.dlrm_linear_fwd_workspace_size(x, w)), _ws(dl.dlrm_linear_bwd_workspace_size(y, x, w))
    dims = [13, 512, 256, 128]
    mx, mw = _rand(g, B, 13), _rand(g, 200000, std=0.05, dtype="f16")
    mb, mo = _rand(g, 1024), torch.zeros(B, 128, device=dev()).half()
    ms = _ws(dl.dlrm_bottom_mlp_workspace_size(B, dims))
    return {
        "interaction": (lambda s: dl.dlrm_interact_fwd(dense, pooled, F, D, B, out, P, stream=s), [out]),
        "interaction backward": (lambda s: dl.dlrm_interact_bwd_f16(go, dense, pooled, F, D, B, P, gd, gp, stream=s), [gd, gp]),
        "bottom MLP": (lambda s: dl.dlrm_bottom_mlp_fwd(mx, dims, mw, mb, mo, ms, stream=s), [mo]),
        "layer": (lambda s: dl.dlrm_linear_fwd(x, w, None, None, y, workspace=wf, stream=s), [y]),
        "gradient": (lambda s: dl.dlrm_linear_bwd(dy, x, w, None, dx, dw, db, workspace=wb, stream=s), [dx, dw, db]),
        "mixture": (lambda s: m.run(s), [m.y, m.ids, m.probs]),
    }


@pytest.mark.parametrize("name", ["interaction", "interaction backward", "bottom MLP", "layer", "gradient", "mixture"])
def test_first_call_of_a_thread(cuda_lib, name):
    call, outputs = _cases(cuda_lib)[name]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(stream)
    torch.cuda.synchronize()
    want = [t.clone() for t in outputs]
    for t in outputs:
        t.zero_()
    torch.cuda.synchronize()
    _in_new_thread(lambda: call(stream))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outputs, want))
    assert any(bool((t != 0).any()) for t in want)


def test_threads_at_once(cuda_lib):
    """Four threads, each with its stream and buffers, have the bits of calls one after another."""
    def work(seed):
        g = torch.Generator().manual_seed(seed)
        m = Mixture(cuda_lib, ("f32", "f16", "bf16", "f16")[seed], 128 + 8 * seed, 64, T=3 + seed, seed=seed)
        x, w = _rand(g, 300, 64, dtype="f16"), _rand(g, 96 + seed, 64, std=0.1, dtype="f16")
        dy, y = _rand(g, 300, 96 + seed, dtype="f16"), torch.empty(300, 96 + seed, dtype=torch.float16, device=dev())
        return m, x, w, dy, y, torch.empty_like(x), torch.empty_like(w), torch.empty(96 + seed, device=dev())

    def step(state, stream):
        m, x, w, dy, y, dx, dw, db = state
        m.run(stream)
        cuda_lib.dlrm_linear_fwd(x, w, None, None, y, act=2, workspace=state_ws[id(m)][0], stream=stream)
        cuda_lib.dlrm_linear_bwd(dy, x, w, y, dx, dw, db, act=2, workspace=state_ws[id(m)][1], stream=stream)

    def results(state):
        return state[0].outputs() + [t.clone() for t in state[4:]]

    states = [work(s) for s in range(4)]
    state_ws = {id(s[0]): (_ws(cuda_lib.dlrm_linear_fwd_workspace_size(s[1], s[2])),
                           _ws(cuda_lib.dlrm_linear_bwd_workspace_size(s[3], s[1], s[2], act=2))) for s in states}
    want = []
    for s in states:
        step(s, None)
        want.append(results(s))
    for s in states:
        for t in (s[0].y, *s[4:]):
            t.zero_()
    torch.cuda.synchronize()
    errors = []

    def run(s):
        try:
            stream = torch.cuda.Stream()
            for _ in range(50):
                step(s, stream)
            stream.synchronize()
        except Exception as e:      # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(s,)) for s in states]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for s, w in zip(states, want):
        assert all(torch.equal(a, b) for a, b in zip(results(s), w))
