"""A residual block of experts in training: the norm before the block, the experts' choice and order, the
rows' way to their experts and back, and the norm after it with a gate and a residual scale, fused with the
next block's norm.

    x --------------------------------------------------------------+-> r
    h = norm(x) -> router -> choice -> order -> experts -> combine -+-> norm, gate, scale;  next h = norm(r)

Every product, norm, choice, sort, gather and gradient is a kernel of the library; torch holds the memory
and applies SGD.  With ``bits8`` what the experts' gradients need is kept in 8 bits between the passes.
Run:  python examples/train_mixture.py [steps]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dlrm_embeddings_dot_gb300 as dl  # noqa: E402

DEV = "cuda:0"
ACT = dl.DLRM_ACT_GELU
NORM = dict(norm=dl.DLRM_NORM_RMS, gate_act=dl.DLRM_GATE_SIGMOID)


def _space(n):
    return torch.empty(n, dtype=torch.uint8, device=DEV) if n else None


def _linear(x, w, bias, act=dl.DLRM_ACT_NONE, y=None, pre=None):
    y = torch.empty(x.shape[0], w.shape[0], dtype=x.dtype, device=DEV) if y is None else y
    dl.dlrm_linear_fwd(x, w, bias, None, y, pre=pre, act=act, workspace=_space(dl.dlrm_linear_fwd_workspace_size(x, w)))
    return y


def _linear_grad(gy, x, w, gx, gw, gb, pre=None, act=dl.DLRM_ACT_NONE):
    """x and pre: tensors, or in 8 bits pairs (bytes, exponents)."""
    if isinstance(x, tuple):
        zq, ze = pre if pre is not None else (None, None)
        ws = _space(dl.dlrm_linear_bwd8_workspace_size(gy, x[0], w, act=act))
        dl.dlrm_linear_bwd8(gy, *x, w, zq, ze, gx, gw, gb, act=act, workspace=ws)
    else:
        ws = _space(dl.dlrm_linear_bwd_workspace_size(gy, x, w, act=act))
        dl.dlrm_linear_bwd(gy, x, w, pre, gx, gw, gb, act=act, workspace=ws)


def _pack(x):
    q = torch.empty(x.shape, dtype=torch.uint8, device=DEV)
    e = torch.empty(x.shape[0], (x.shape[1] + 31) // 32, dtype=torch.uint8, device=DEV)
    dl.dlrm_pack8(x, q, e)
    return q, e


def _rows(kept, a, b):
    return tuple(t[a:b] for t in kept) if isinstance(kept, tuple) else kept[a:b]


class MixtureBlock:
    """(x, h) -> (r, next h), with h the norm of x; a block of width H, E experts of `hidden`, k of them a token."""

    def __init__(self, width, hidden, experts, k, dtype=torch.float32, bits8=False, seed=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device=DEV) / shape[-1] ** 0.5).to(dtype)

        self.k, self.bits8 = k, bits8
        self.p = dict(router=weight(experts, width), gate=weight(1, width), w1=weight(experts, hidden, width),
                      b1=torch.zeros(experts, hidden, device=DEV), w2=weight(experts, width, hidden),
                      w_post=torch.ones(width, device=DEV), scale=torch.full((width,), 0.5, device=DEV),
                      w_next=torch.ones(width, device=DEV))
        self.g = {n: torch.empty_like(v) for n, v in self.p.items()}

    def forward(self, x, h):
        p, (T, H), k = self.p, x.shape, self.k
        E, hidden = p["w1"].shape[:2]

        def new(*shape, dtype=x.dtype):
            return torch.empty(*shape, dtype=dtype, device=DEV)

        logits, gate = _linear(h, p["router"], None), _linear(h, p["gate"], None)
        ids, probs = new(T, k, dtype=torch.int32), new(T, k, dtype=torch.float32)
        dl.dlrm_route_fwd(logits, ids, probs)
        offsets, slots = new(E + 1, dtype=torch.int32), new(T, k, dtype=torch.int32)
        dl.dlrm_expert_sort(ids, E, offsets, slots, workspace=_space(dl.dlrm_expert_sort_workspace_size(ids, E)))
        xs, z, a, ys = new(T * k, H), new(T * k, hidden), new(T * k, hidden), new(T * k, H)
        dl.dlrm_dispatch_fwd(h, slots, xs)
        at = offsets.tolist()               # the layers' sizes are the host's
        for e in range(E):
            rows = slice(at[e], at[e + 1])
            if rows.start < rows.stop:
                _linear(xs[rows], p["w1"][e], p["b1"][e], ACT, y=a[rows], pre=z[rows])
                _linear(a[rows], p["w2"][e], None, y=ys[rows])
        m = new(T, H)
        dl.dlrm_combine_fwd(ys, slots, probs, None, m)
        r, h_next, stats = new(T, H), new(T, H), new(T, 4, dtype=torch.float32)
        dl.dlrm_block_norm_fwd(m, gate, x, p["w_post"], None, p["scale"], p["w_next"], None, r, h_next, stats, **NORM)
        if self.bits8:
            n = at[E]
            xs, z, a = _pack(xs[:n]), _pack(z[:n]), _pack(a[:n])
        self.kept = dict(h=h, gate=gate, ids=ids, probs=probs, slots=slots, at=at, xs=xs, z=z, a=a, ys=ys, m=m, r=r, stats=stats)
        return r, h_next

    def backward(self, grad_r, grad_h):
        """Gradients of x (the residual's way) and h; the parameters' go to self.g."""
        p, g, s = self.p, self.g, self.kept
        T, H = s["m"].shape
        E = p["w1"].shape[0]
        gx, gm, ggate = torch.empty_like(s["m"]), torch.empty_like(s["m"]), torch.empty_like(s["gate"])
        dl.dlrm_block_norm_bwd(grad_r, grad_h, s["m"], s["gate"], s["r"], s["stats"], p["w_post"], None, p["scale"], p["w_next"],
                               gm, ggate, gx, g["w_post"], None, g["scale"], g["w_next"], None,
                               workspace=_space(dl.dlrm_block_norm_bwd_workspace_size(s["m"])), **NORM)
        gys, gprobs = torch.empty_like(s["ys"]), torch.empty_like(s["probs"])
        dl.dlrm_combine_bwd(gm, s["ys"], s["slots"], s["probs"], gys, gprobs)
        ga = torch.empty(T * self.k, p["w1"].shape[1], dtype=gm.dtype, device=DEV)
        gxs = torch.empty_like(gys)
        for e in range(E):
            a, b = s["at"][e], s["at"][e + 1]
            if a == b:
                for n in ("w1", "b1", "w2"):
                    g[n][e].zero_()
                continue
            _linear_grad(gys[a:b], _rows(s["a"], a, b), p["w2"][e], ga[a:b], g["w2"][e], None)
            _linear_grad(ga[a:b], _rows(s["xs"], a, b), p["w1"][e], gxs[a:b], g["w1"][e], g["b1"][e], pre=_rows(s["z"], a, b),
                         act=ACT)
        gh, more = torch.empty_like(gm), torch.empty_like(gm)
        dl.dlrm_dispatch_bwd(gxs, s["slots"], gh)
        glogits = torch.empty(T, E, dtype=gm.dtype, device=DEV)
        dl.dlrm_route_bwd(gprobs, s["ids"], s["probs"], glogits)
        for gy, n in ((glogits, "router"), (ggate, "gate")):
            _linear_grad(gy, s["h"], p[n], more, g[n], None)
            gh += more
        return gx, gh

    def step(self, lr):
        for n, v in self.p.items():
            v.sub_(lr * self.g[n])


def first_norm(x):
    """The first block's h, and what its gradient needs."""
    h, stats = torch.empty_like(x), torch.empty(x.shape[0], 4, device=DEV)
    dl.dlrm_block_norm_fwd(None, None, x, None, None, None, None, None, None, h, stats, **NORM)
    return h, stats


def first_norm_grad(x, stats, grad_x, grad_h):
    """grad_x and the way through the norm."""
    out = torch.empty_like(x)
    dl.dlrm_block_norm_bwd(grad_x, grad_h, None, None, x, stats, None, None, None, None, None, None, out, None, None, None, None,
                           None, **NORM)
    return out


def train(steps=30, tokens=512, width=128, bits8=True, seed=0):
    """Two blocks learn a fixed linear rule of their input; returns the losses."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(tokens, width, generator=g, device=DEV)
    target = x @ torch.randn(width, width, generator=g, device=DEV) / width**0.5
    blocks = [MixtureBlock(width, 96, 8, 2, bits8=bits8, seed=seed + i) for i in range(2)]
    losses = []
    for _ in range(steps):
        h, _ = first_norm(x)
        r = x
        for b in blocks:
            r, h = b.forward(r, h)
        losses.append(((h - target) ** 2).mean())
        gr, gh = torch.zeros_like(r), 2 * (h - target) / tokens
        for b in reversed(blocks):
            gr, gh = b.backward(gr, gh)
            b.step(0.02)
    return [float(v) for v in losses]


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 30
    for bits8 in (False, True):
        losses = train(steps, bits8=bits8)
        print(f"{'8-bit' if bits8 else 'fp32 '} activations: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")


if __name__ == "__main__":
    main()
