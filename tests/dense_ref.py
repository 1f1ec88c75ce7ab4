"""Plain 64-bit forms of the dense network's operators for its tests, and the error bounds
they are held to.

Bounds, from the formulas (u = half an ulp of the output type, relative; A = the same
expression on absolute values):
  * a product of length L summed in fp32 in any order, terms cut instead of rounded: (L + 8) 2^-23 A;
    the three-part form of fp32 leaves out terms below 2^-22 A, within the same bound
  * an activation or its slope in fp32: 2^-20 of its largest factor; it stretches an error of z
    by at most 1.13
  * each value rounded to the type: u of its size, and half the least subnormal of fp16
  * the gradient products take dZ rounded to the type: u A more
"""

import math

import numpy as np
import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0**-24, "f16": 2.0**-11, "bf16": 2.0**-8}
TINY = {"f32": 2.0**-149, "f16": 2.0**-24, "bf16": 2.0**-133}
ACT = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}


def philox(counter, key):
    """Philox4x32-10 with Python integers (Salmon, Moraes, Dror, Shaw, SC 2011)."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p):
    return int(math.floor(65536 * p + 0.5))


def numbers(seed, offset, M, N):
    """The 16-bit number of every element, uint16 [M][N] (vectorised over elements)."""
    seed, offset = seed % 2**64, offset % 2**64
    groups = (N + 7) // 8
    c = [np.tile(np.arange(groups, dtype=np.uint64), M), np.repeat(np.arange(M, dtype=np.uint64), groups),
         np.full(M * groups, offset & 0xFFFFFFFF, np.uint64), np.full(M * groups, offset >> 32, np.uint64)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    low, s32 = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> s32) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> s32) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    out = np.empty((M, groups, 8), np.uint16)
    for j in range(4):
        w = c[j].reshape(M, groups)
        out[:, :, 2 * j] = (w & np.uint64(0xFFFF)).astype(np.uint16)
        out[:, :, 2 * j + 1] = (w >> np.uint64(16)).astype(np.uint16)
    return out.reshape(M, groups * 8)[:, :N]


def keep_scale(seed, offset, M, N, p):
    """(kept bool [M][N], scale) of the dropout of an M x N matrix."""
    t = threshold(p)
    return torch.from_numpy(numbers(seed, offset, M, N) >= t), 65536.0 / (65536 - t)


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def slope(z, name):
    if name == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), torch.ones_like(z))
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def linear_fwd(x, w, b, res, name, kept=None, scale=1.0):
    """(y, z, bound of y, bound of z) without the rounding to the type; inputs in 64 bits."""
    K = x.shape[1]
    z = x @ w.t()
    a = x.abs() @ w.abs().t()
    if b is not None:
        z, a = z + b, a + b.abs()
    ez = (K + 8) * 2.0**-23 * a
    y, ey = act(z, name), 1.13 * ez + 2.0**-20 * z.abs()
    if kept is not None:
        y, ey = torch.where(kept, y * scale, torch.zeros_like(y)), torch.where(kept, ey * scale, torch.zeros_like(ey))
    if res is not None:
        ey = ey + 2.0**-23 * (y.abs() + res.abs())
        y = y + res
    return y, z, ey, ez


def linear_bwd(dy, x, w, z, name, u, kept=None, scale=1.0):
    """{gradient: (value, bound)} without the last rounding; inputs in 64 bits."""
    M, N = dy.shape
    g = dy if kept is None else torch.where(kept, dy * scale, torch.zeros_like(dy))
    s = slope(z, name) if name != "none" else torch.ones_like(g)
    dz = g * s
    size = g.abs() * 1.2
    edz = 2.0**-20 * size if name != "none" else 2.0**-23 * size
    dx, dw = dz @ w, dz.t() @ x
    one = dz.abs() * (u + 2.0**-23) + edz + (2.0**-25 if u == U["f16"] else 0.0)   # dZ rounded to the type
    return {"dx": (dx, one @ w.abs() + (N + 8) * 2.0**-23 * (size @ w.abs())),
            "dw": (dw, one.t() @ x.abs() + (M + 8) * 2.0**-23 * (size.t() @ x.abs())),
            "db": (dz.sum(0), edz.sum(0) + (M + 8) * 2.0**-23 * size.sum(0))}


def assert_close(got, ref, bound, dtype, what=""):
    """|got - ref| <= bound + rounding to the type, elementwise, in 64 bits."""
    got, ref = got.double().cpu(), ref.cpu()
    tol = bound.cpu() * (1 + U[dtype]) + U[dtype] * ref.abs() + TINY[dtype] + 1e-300
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off; first at {i}: got "
                             f"{got[tuple(i)].item()!r}, ref {ref[tuple(i)].item()!r}, bound {tol[tuple(i)].item()!r}")


def moe_route(logits, k):
    """(ids, probs): the k largest logits of each row, ties to the lower index, and their softmax."""
    order = torch.argsort(-logits, dim=1, stable=True)[:, :k]
    return order, torch.softmax(torch.gather(logits, 1, order), 1)


def moe(x, wr, w1, w2, res, ids, name, gated, u):
    """(y, bound of y, probs) for given choices; inputs in 64 bits."""
    T, H = x.shape
    E, I = w2.shape[0], w2.shape[2]
    logits = x @ wr.t()
    probs = torch.softmax(torch.gather(logits, 1, ids), 1)
    el = (H + 8) * 2.0**-23 * (x.abs() @ wr.abs().t())
    ep = 2 * torch.gather(el, 1, ids).max(1, keepdim=True).values * probs + 2.0**-20 * probs
    y, ey = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            z, a = w1[e] @ x[t], w1[e].abs() @ x[t].abs()
            ez = (H + 8) * 2.0**-23 * a
            h, eh = act(z[:I], name), 1.13 * ez[:I] + 2.0**-20 * z[:I].abs()
            if gated:
                eh = eh * (z[I:].abs() + ez[I:]) + h.abs() * ez[I:]
                h = h * z[I:]
            ph, eph = probs[t, j] * h, probs[t, j] * eh + ep[t, j] * (h.abs() + eh)
            eph = eph + (u + 2.0**-22) * (ph.abs() + eph) + (2.0**-25 if u == 2.0**-11 else 0.0)
            y[t] += w2[e] @ ph
            ey[t] += w2[e].abs() @ eph + (ids.shape[1] * I + 8) * 2.0**-23 * (w2[e].abs() @ (ph.abs() + eph))
    if res is not None:
        ey = ey + 2.0**-23 * (y.abs() + res.abs())
        y = y + res
    return y, ey, probs, ep
