"""A small DLRM end to end on one GPU: training steps of the whole network, then a request
scored through a mixture-of-experts head.

    dense features -> bottom MLP -+
    categorical    -> lookup     -+-> dot interaction -> top MLP (dropout, a skip connection) -> logit

Every matrix product, activation, dropout, lookup, interaction, gradient and table update is a
kernel of the library; torch holds the memory, applies SGD to the small dense weights and
computes the loss's slope.  Run:  python examples/train_and_score.py [steps]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dlrm_embeddings_dot_gb300 as dl  # noqa: E402

DEV = "cuda:0"
TABLES, WIDTH, ROWS, BATCH = 8, 128, 500, 1024
COLUMNS = 164        # WIDTH + 9 * 8 / 2 interaction columns
LR, DROPOUT = 0.05, 0.1


class Layer:
    """A dense layer with its gradients, buffers and workspaces, for a fixed batch."""

    def __init__(self, rows, n_in, n_out, act, p=0.0, gen=None):
        lim = (6.0 / (n_in + n_out)) ** 0.5
        self.w = (torch.rand(n_out, n_in, generator=gen, device=DEV) * 2 - 1) * lim
        self.b = torch.zeros(n_out, device=DEV)
        self.act, self.p = act, p
        self.y, self.z = (torch.empty(rows, n_out, device=DEV) for _ in range(2))
        self.dx = torch.empty(rows, n_in, device=DEV)
        self.dw, self.db = torch.empty_like(self.w), torch.empty_like(self.b)
        x = torch.empty(rows, n_in, device=DEV)
        self.ws = torch.empty(max(dl.dlrm_linear_fwd_workspace_size(x, self.w),
                                  dl.dlrm_linear_bwd_workspace_size(self.y, x, self.w, act=act, p=p), 256),
                              dtype=torch.uint8, device=DEV)

    def forward(self, x, residual=None, rng=None, train=True):
        p = self.p if train else 0.0
        dl.dlrm_linear_fwd(x, self.w, self.b, residual, self.y, pre=self.z, act=self.act, p=p, rng=rng, workspace=self.ws)
        self.x, self.rng = x, rng
        return self.y

    def backward(self, dy):
        dl.dlrm_linear_bwd(dy, self.x, self.w, self.z, self.dx, self.dw, self.db, act=self.act, p=self.p, rng=self.rng,
                           workspace=self.ws)
        return self.dx

    def step(self):
        self.w.sub_(LR * self.dw)
        self.b.sub_(LR * self.db)


class Model:
    def __init__(self, seed=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        F, D, B = TABLES, WIDTH, BATCH
        self.tables = torch.empty(F * ROWS, D, device=DEV)
        dl.dlrm_synth_fill_uniform(self.tables, seed, 0)
        self.row_base = torch.arange(0, F * ROWS + 1, ROWS, device=DEV)
        self.bottom = [Layer(B, 13, 64, dl.DLRM_ACT_RELU, gen=g), Layer(B, 64, D, dl.DLRM_ACT_RELU, gen=g)]
        self.top = [Layer(B, COLUMNS, 256, dl.DLRM_ACT_GELU, DROPOUT, gen=g),
                    Layer(B, 256, 256, dl.DLRM_ACT_GELU, DROPOUT, gen=g),   # with a skip connection
                    Layer(B, 256, 1, dl.DLRM_ACT_NONE, gen=g)]
        self.pooled, self.dpooled = (torch.empty(B, F, D, device=DEV) for _ in range(2))
        self.inter = torch.empty(B, COLUMNS, device=DEV)
        self.ddense = torch.empty(B, D, device=DEV)
        self.ws = torch.empty(dl.dlrm_emb_bwd_sgd_workspace_size(B * F, D, F * ROWS), dtype=torch.uint8, device=DEV)
        # one generator state a dropout layer: (seed, offset); a step advances the offsets
        self.rng = [torch.tensor([seed + 17 * i, 0], device=DEV) for i in range(2)]

    def forward(self, dense, indices, offsets, train=True):
        h = self.bottom[1].forward(self.bottom[0].forward(dense))
        dl.dlrm_emb_interact_fwd_train(self.tables, self.row_base, TABLES, WIDTH, BATCH, indices, offsets, h, self.pooled,
                                       self.inter, COLUMNS)
        t = self.top[0].forward(self.inter, rng=self.rng[0], train=train)
        t = self.top[1].forward(t, residual=t, rng=self.rng[1], train=train)
        return self.top[2].forward(t)

    def backward(self, dlogit, indices, offsets):
        dskip = self.top[2].backward(dlogit)
        dt = self.top[1].backward(dskip)
        dinter = self.top[0].backward(dt.add_(dskip))       # the residual's gradient is its layer's own
        dl.dlrm_interact_bwd(dinter, self.bottom[1].y, self.pooled, TABLES, WIDTH, BATCH, COLUMNS, self.ddense, self.dpooled)
        self.bottom[0].backward(self.bottom[1].backward(self.ddense))
        dl.dlrm_emb_bwd_sgd(self.tables, self.row_base, TABLES * ROWS, TABLES, WIDTH, BATCH, indices, offsets, self.dpooled,
                            LR, self.ws)
        for layer in self.bottom + self.top:
            layer.step()
        for r in self.rng:
            r[1] += 1


def train(steps=60, seed=0):
    """Trains on labels that follow a fixed rule; returns (model, losses)."""
    model = Model(seed)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 1)
    dense = torch.randn(BATCH, 13, generator=g, device=DEV)
    indices = torch.randint(0, ROWS, (TABLES * BATCH,), generator=g, device=DEV, dtype=torch.int32)
    offsets = torch.arange(TABLES * BATCH + 1, device=DEV, dtype=torch.int32)
    label = ((dense[:, 0] + 0.5 * dense[:, 1] + (indices[:BATCH] % 2) - 0.5) > 0).float()[:, None]
    losses = []
    for _ in range(steps):
        logit = model.forward(dense, indices, offsets)
        prob = torch.sigmoid(logit)
        losses.append(torch.nn.functional.binary_cross_entropy(prob, label))
        model.backward((prob - label) / BATCH * 8, indices, offsets)
    return model, [float(v) for v in losses]


def score(model, experts=8, hidden=128, top_k=2, requests=4):
    """Scores a few interaction rows through a gated mixture with a skip connection, then the logit layer."""
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    x = model.top[1].y[:requests].contiguous()
    H = x.shape[1]
    w_router = torch.randn(experts, H, generator=g, device=DEV) / H**0.5
    w1 = torch.randn(experts, 2 * hidden, H, generator=g, device=DEV) / H**0.5
    w2 = torch.randn(experts, H, hidden, generator=g, device=DEV) / hidden**0.5
    y, probs = torch.empty_like(x), torch.empty(requests, top_k, device=DEV)
    ids = torch.empty(requests, top_k, dtype=torch.int32, device=DEV)
    ws = torch.empty(dl.dlrm_moe_fwd_workspace_size(x, w_router, w1, w2, top_k), dtype=torch.uint8, device=DEV)
    dl.dlrm_moe_fwd(x, w_router, w1, w2, x, y, ids, probs, act=dl.DLRM_ACT_SILU, gated=True, workspace=ws)
    last = model.top[2]
    logit = torch.empty(requests, 1, device=DEV)
    dl.dlrm_linear_fwd(y, last.w, last.b, None, logit)      # few rows: no workspace
    return logit, ids, probs


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 60
    model, losses = train(steps)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps of {BATCH} samples")
    logit, ids, probs = score(model)
    for i in range(logit.shape[0]):
        chosen = ", ".join(f"{e}: {p:.2f}" for e, p in zip(ids[i].tolist(), probs[i].tolist()))
        print(f"request {i}: logit {float(logit[i]):+.3f} through experts {chosen}")


if __name__ == "__main__":
    main()
