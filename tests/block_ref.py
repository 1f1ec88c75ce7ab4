"""Plain 64-bit forms of the residual blocks' operators (include/dlrm_block.h) for their tests, and the
error bounds they are held to.

Bounds, from the formulas (u = half an ulp of the output type, relative; e_v = the bound of a value v):
  * a sum of L terms in fp32 in any order: (L + 8) 2^-23 of the sum of their sizes
  * a product, sum or fused pair of values: 2^-22 of the sizes that enter it, next to what it inherits
  * 1 / sqrt(s): half the relative bound of s, and 2^-22
  * a gate or its slope: 2^-19 of its largest factors (the exponential and reciprocal of 2-byte types are
    within 2^-21; fp32's are better)
Each output is then rounded once: u of its size (``dense_ref.assert_close`` adds it).
"""

import torch

SUM, OP = 2.0**-23, 2.0**-22
GATES = {"raw": 0, "sigmoid": 1, "silu": 2}


def gate(g, name):
    s = torch.sigmoid(g)
    return {"raw": g, "sigmoid": s, "silu": g * s}[name]


def gate_slope(g, name):
    s = torch.sigmoid(g)
    return {"raw": torch.ones_like(g), "sigmoid": s * (1 - s), "silu": s * (1 + g * (1 - s))}[name]


def norm(v, e, layer, eps):
    """(mean, rstd, x, bound of x) of rows v whose values are known to e."""
    n = v.shape[1]
    zero = torch.zeros_like(v[:, :1])
    m = v.mean(1, keepdim=True) if layer else zero
    em = e.mean(1, keepdim=True) + (n + 8) * SUM * v.abs().mean(1, keepdim=True) if layer else zero
    d = v - m
    ed = e + em + OP * (v.abs() + m.abs())
    ss = (d * d).mean(1, keepdim=True)
    ess = (2 * d.abs() * ed + ed * ed).mean(1, keepdim=True) + (n + 8) * SUM * ss
    s = (ss + eps) ** -0.5
    rel = ess / (ss + eps) + OP
    return m, s, d * s, s * ed * (1 + rel) + (d * s).abs() * rel


def forward(y, g, res, w_post, b_post, scale, w_pre, b_pre, layer, gate_act, eps, want_h=True):
    """{name: (value, bound)} of r, h and the four statistics; inputs in 64 bits or None."""
    like = y if y is not None else res
    one, zero = torch.ones(like.shape[1], dtype=torch.float64), torch.zeros_like(like)
    r = zero if res is None else res
    er, out = zero, {}
    if y is not None:
        m, s, x, ex = norm(y, zero, layer, eps)
        w, b, c = (one if w_post is None else w_post), (0 * one if b_post is None else b_post), (one if scale is None else scale)
        u = x * w + b
        eu = ex * w.abs() + OP * ((x * w).abs() + b.abs())
        q = torch.ones_like(zero) if g is None else gate(g, gate_act)
        eq = 0 * zero if g is None or gate_act == "raw" else 2.0**-19 * (q.abs() + 1e-30)
        t = c * q * u
        er = c.abs() * (eu * (q.abs() + eq) + u.abs() * eq) + OP * (t.abs() * 2 + r.abs())
        r = r + t
        out["r"], out["y_stats"] = (r, er), (m, s)
    if want_h:
        m, s, x, ex = norm(r, er, layer, eps)
        w, b = (one if w_pre is None else w_pre), (0 * one if b_pre is None else b_pre)
        out["h"] = (x * w + b, ex * w.abs() + OP * ((x * w).abs() + b.abs()))
        out["r_stats"] = (m, s)
    return out


def _norm_grad(d, ed, x, ex, s, layer):
    n = d.shape[1]
    c0, a0 = (d * x).mean(1, keepdim=True), (d * x).abs().mean(1, keepdim=True)
    e0 = (ed * x.abs() + d.abs() * ex + ed * ex).mean(1, keepdim=True) + (n + 8) * SUM * a0
    c1, e1 = 0 * c0, 0 * c0
    if layer:
        c1 = d.mean(1, keepdim=True)
        e1 = ed.mean(1, keepdim=True) + (n + 8) * SUM * d.abs().mean(1, keepdim=True)
    v = s * (d - c1 - x * c0)
    e = s * (ed + e1 + x.abs() * e0 + ex * (c0.abs() + e0)) + 4 * OP * s * (d.abs() + c1.abs() + (x * c0).abs())
    return v, e


def backward(gr, gh, y, g, r, stats, w_post, b_post, scale, w_pre, layer, gate_act):
    """{gradient: (value, bound)}; stats as they were given to the call."""
    like = gr if gr is not None else gh
    M, N = like.shape
    one, zero = torch.ones(N, dtype=torch.float64), torch.zeros_like(like)
    out = {}

    def hat(v, m, s):
        x = (v - m) * s
        return x, s.abs() * OP * (v.abs() + m.abs()) + OP * x.abs()

    def rows(v, e):
        return v.sum(0), e.sum(0) + (M + 8) * SUM * v.abs().sum(0)

    dr, er = (zero if gr is None else gr), zero
    if gh is not None:
        x, ex = hat(r, stats[:, 2:3], stats[:, 3:4])
        w = one if w_pre is None else w_pre
        d = gh * w
        v, e = _norm_grad(d, OP * d.abs(), x, ex, stats[:, 3:4], layer)
        dr, er = dr + v, e + OP * (dr.abs() + v.abs())
        out["w_pre"], out["b_pre"] = rows(gh * x, gh.abs() * ex + OP * (gh * x).abs()), rows(gh, 0 * gh)
    out["residual"] = (dr, er)
    if y is not None:
        x, ex = hat(y, stats[:, 0:1], stats[:, 1:2])
        w, b, c = (one if w_post is None else w_post), (0 * one if b_post is None else b_post), (one if scale is None else scale)
        q, k = (torch.ones_like(zero), 0 * zero) if g is None else (gate(g, gate_act) + zero, gate_slope(g, gate_act) + zero)
        rough = 0.0 if g is None or gate_act == "raw" else 2.0**-19
        eq = rough * q.abs()
        # the slopes' factors: sigmoid s (1 - s), silu s (1 + g (1 - s)); each factor to 2^-19 of its terms
        ek = 0 * zero
        if g is not None and gate_act != "raw":
            s = torch.sigmoid(g)
            ek = rough * (s * (1 + g.abs()) + k.abs()) * 2 + zero
        a = dr * q
        ea = er * (q.abs() + eq) + dr.abs() * eq + OP * a.abs()
        d = a * c * w
        ed = ea * (c * w).abs() + 2 * OP * d.abs()
        out["y"] = _norm_grad(d, ed, x, ex, stats[:, 1:2], layer)
        u = x * w + b
        eu = ex * w.abs() + 2 * OP * ((x * w).abs() + b.abs())
        s0, s1 = rows(a * x, ea * x.abs() + (a.abs() + ea) * ex + OP * (a * x).abs()), rows(a, ea)
        out["w_post"] = (c * s0[0], c.abs() * (s0[1] + OP * s0[0].abs()))
        out["b_post"] = (c * s1[0], c.abs() * (s1[1] + OP * s1[0].abs()))
        out["scale"] = (w * s0[0] + b * s1[0], w.abs() * s0[1] + b.abs() * s1[1] + OP * ((w * s0[0]).abs() + (b * s1[0]).abs()))
        if g is not None:
            t = dr * c * u
            et = c.abs() * (er * (u.abs() + eu) + dr.abs() * eu) + 2 * OP * (dr.abs() * c.abs() * ((x * w).abs() + b.abs()))
            if g.shape[1] == 1:
                k, ek = k[:, :1], ek[:, :1]
                et = et.sum(1, keepdim=True) + (N + 8) * SUM * t.abs().sum(1, keepdim=True)
                t = t.sum(1, keepdim=True)
            out["gate"] = (t * k, et * (k.abs() + ek) + t.abs() * ek + OP * (t * k).abs())
    return out


# ------------------------------------------------------------------------------------------- experts
def route(logits, k):
    """(ids, probs): NaN largest, -infinity closed, ties to the lower index."""
    T, E = logits.shape
    ids, probs = torch.full((T, k), -1, dtype=torch.int64), torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        row = logits[t].tolist()
        order = sorted((e for e in range(E) if not row[e] == -float("inf")),
                       key=lambda e: (-float("inf") if row[e] != row[e] else -row[e], row[e] == row[e], e))[:k]
        for j, e in enumerate(order):
            ids[t, j] = e
        if order:
            top = logits[t, order]
            w = torch.exp(top - top[0])
            probs[t, :len(order)] = w / w.sum()
    return ids, probs


def sort(ids, E):
    """(offsets, slots, order) of a list of lists of choices."""
    flat = [e for row in ids for e in row]
    k = len(ids[0]) if ids else 1
    order = sorted((c for c, e in enumerate(flat) if 0 <= e < E), key=lambda c: (flat[c], c))
    slots = [-1] * len(flat)
    for place, c in enumerate(order):
        slots[c] = place
    offsets = [sum(1 for e in flat if 0 <= e < b) for b in range(E + 1)]
    return offsets, [slots[i:i + k] for i in range(0, len(flat), k)], order + [-1] * (len(flat) - len(order))


# ------------------------------------------------------------------------------------------- 8 bits
def code_values():
    """The 256 values of the 8-bit floats."""
    out = []
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        v = (1 + m / 8) * 2.0**(e - 7) if e else m / 8 * 2.0**-6
        out.append(float("nan") if b & 127 == 127 else -v if b & 128 else v)
    return torch.tensor(out, dtype=torch.float64)


def pack8(x):
    """(bytes, exponents) by search over the format's values; signs of zeros as the input's."""
    M, N = x.shape
    v = torch.zeros(M, -(-N // 32) * 32, dtype=torch.float64)
    v[:, :N] = x.double()
    v = v.view(M, -1, 32)
    finite = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v))
    top = finite.amax(2)
    e = torch.zeros_like(top, dtype=torch.int64)
    for i in range(254, -1, -1):     # the least that is enough
        e = torch.where(top <= 448 * 2.0**(i - 127), i, e)
    values = code_values()[:127]
    middle = (values[1:] + values[:-1]) / 2
    a = (finite * torch.exp2(127.0 - e)[:, :, None]).reshape(-1)
    lo, hi = torch.searchsorted(middle, a), torch.searchsorted(middle, a, right=True)
    q = torch.where((lo != hi) & (lo % 2 == 1), hi, lo).view(v.shape)
    q = q + 128 * torch.signbit(v)
    q = torch.where(torch.isfinite(v), q, 127)
    return q.view(M, -1)[:, :N], e


def unpack8(q, e, largest):
    v = code_values()[q.long()] * torch.exp2(e.double() - 127).repeat_interleave(32, 1)[:, :q.shape[1]]
    return torch.where(v.abs() > largest, torch.copysign(torch.tensor(largest, dtype=torch.float64), v), v)
