"""Cases of the dense network's residual blocks in training and serving: the norms after and before a block with its gate
and residual scale, the choice of experts and the order of the tokens by expert, the way of the tokens to their experts
and back, and activations kept in 8 bits with the layer gradient that reads them.

``run`` computes each in its plain form (elementary torch operations in 32 bits, rounded once at the end) or, with
``own`` set, through the library's entry points.  ``exact`` computes the same outputs in 64 bits."""

import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
LARGEST = {"f32": 3.3895313892515355e38, "f16": 65504.0, "bf16": 3.3895313892515355e38}   # of a value read from 8 bits
ACTS = ("none", "relu", "gelu", "silu")
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ cases
def _norm(name, m, n, dtype, kind, gate, backward=False, per_row=False, pre=True, post=True, extras=True, pad=0):
    """kind: rms or layer; gate: none (absent), raw, sigmoid or silu, one value an element or (per_row) a row; post and
    pre: the norm after the block and the one before the next; extras: biases, residual scale and both paths' gradients."""
    return {"name": name, "op": "norm", "m": m, "n": n, "dtype": dtype, "kind": kind, "gate": gate, "backward": backward,
            "per_row": per_row, "pre": pre, "post": post, "extras": extras, "pad": pad}


def _route(name, t, e, k, dtype, backward=False, masked=0.0):
    return {"name": name, "op": "route", "t": t, "e": e, "k": k, "dtype": dtype, "backward": backward, "masked": masked}


def _experts(name, op, t, h, k, e, dtype, backward=False, residual=False, masked=0.0, pad=0):
    return {"name": name, "op": op, "t": t, "h": h, "k": k, "e": e, "dtype": dtype, "backward": backward,
            "residual": residual, "masked": masked, "pad": pad}


def _keep8(name, m, n, dtype, pad=0):
    return {"name": name, "op": "keep8", "m": m, "n": n, "dtype": dtype, "pad": pad}


def _grad8(name, m, n, k, dtype, act, p=0.0, bias=True, pad=0):
    return {"name": name, "op": "grad8", "m": m, "n": n, "k": k, "dtype": dtype, "act": act, "p": p, "bias": bias, "pad": pad}


def listed():
    return [
        # one candidate scored online, between two blocks over one interaction row; latency
        _norm("norm-1x480", 1, 480, "bf16", "rms", "none", extras=False),
        # the training batch between two gated blocks of the top network's first width
        _norm("norm-65536x1024-gate", 65536, 1024, "bf16", "rms", "silu"),
        # gradients of an fp32 model with an odd width, centred norms and one gate value a sample
        _norm("norm-grad-4099x771", 4099, 771, "f32", "layer", "sigmoid", backward=True, per_row=True),
        # gradients at the training batch, mixed precision
        _norm("norm-grad-65536x1024", 65536, 1024, "f16", "rms", "sigmoid", backward=True),
        # a serving batch's experts and their order
        _route("route-48x64", 48, 64, 6, "f32"),
        # the training batch's experts, and the gradient of the choice; some experts are closed to some samples
        _route("route-65536x64", 65536, 64, 4, "bf16", backward=True, masked=0.1),
        # the training batch's rows to two experts each
        _experts("dispatch-65536x1024", "dispatch", 65536, 1024, 2, 16, "bf16"),
        # back from three experts each to rows of an odd width, fp32, with the skip connection and choices without expert
        _experts("combine-5003x515", "combine", 5003, 515, 3, 7, "f32", residual=True, masked=0.1),
        # gradients of the way back at the training batch
        _experts("combine-grad-65536x512", "combine", 65536, 512, 4, 64, "f16", backward=True),
        # the training batch's activations to 8 bits and back
        _keep8("keep8-65536x1024", 65536, 1024, "bf16"),
        # gradients of a hidden layer at a small training batch, its input and pre-activation in 8 bits
        _grad8("grad8-256x512x1024", 256, 512, 1024, "bf16", "gelu"),
        # gradients of the widest top layer at the training batch, dropout regenerated, activations in 8 bits
        _grad8("grad8-65536x1024x1024", 65536, 1024, 1024, "f16", "relu", p=0.1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "norm", "route", "route", "dispatch", "combine", "combine", "keep8", "grad8", "grad8"))
    dtype = rng.choice(("f32", "f16", "bf16"))
    pad = rng.choice((0, 0, 0, 8, 3))
    backward = rng.random() < 0.5
    masked = rng.choice((0.0, 0.0, 0.1, 0.5))

    def width(lo, hi):   # half of the widths are multiples of 16, as layers' mostly are
        n = _log(rng, lo, hi)
        return min(hi, (n + 15) // 16 * 16) if rng.random() < 0.5 else n

    if op == "norm":
        n = width(1, 8192)
        m = min(_log(rng, 1, 65536), max(1, 2**26 // n))
        gate = rng.choice(("none", "raw", "sigmoid", "silu"))
        parts = rng.choice(("both", "both", "post", "pre"))
        case = _norm("", m, n, dtype, rng.choice(("rms", "layer")), gate if parts != "pre" else "none", backward,
                     gate != "none" and parts != "pre" and rng.random() < 0.3, parts != "post", parts != "pre",
                     rng.random() < 0.7, pad)
    elif op == "route":
        e = _log(rng, 1, 256)
        case = _route("", _log(rng, 1, 65536), e, rng.randint(1, min(e, 8)), dtype, backward, masked)
    elif op in ("dispatch", "combine"):
        h, k, e = width(1, 4096), rng.randint(1, 8), _log(rng, 1, 256)
        t = min(_log(rng, 1, 65536), max(1, 2**27 // (h * k)))
        case = _experts("", op, t, h, k, e, dtype, backward, op == "combine" and not backward and rng.random() < 0.5,
                        masked, pad)
    elif op == "keep8":
        n = width(1, 4096)
        case = _keep8("", min(_log(rng, 1, 65536), max(1, 2**26 // n)), n, dtype, pad)
    else:
        n, k = width(1, 4096), width(1, 4096)
        m = max(1, min(_log(rng, 1, 65536), (2**36 if dtype != "f32" else 2**33) // (n * k)))
        case = _grad8("", m, n, k, dtype, rng.choice(ACTS), rng.choice((0.0, 0.0, 0.1, round(rng.random() * 0.8, 3))),
                      rng.random() < 0.8, pad)
    return {k_: v for k_, v in case.items() if k_ != "name"}


def work(case):
    s, op = SIZE[case["dtype"]], case["op"]
    if op == "norm":
        m, n = case["m"], case["n"]
        gate = 0 if case["gate"] == "none" else 1 if case["per_row"] else n
        if not case["backward"]:   # y, the gate and the residual in; r, h and the rows' statistics out
            rows = n * (1 + case["post"] * 2 + case["pre"]) + gate
            vectors = case["post"] * (1 + 2 * case["extras"]) + case["pre"] * (1 + case["extras"])
            return {"bytes": m * (rows * s + 16) + 4 * n * vectors, "flops": 0}
        # the gradients of r and h, y, the gate and r in; those of y, the gate and the residual out
        both = case["extras"] or not case["pre"]
        rows = n * (both + 2 * case["pre"] + 2 * case["post"] + 1) + 2 * gate
        vectors = case["post"] * (2 + 4 * case["extras"]) + case["pre"] * (2 + case["extras"])
        return {"bytes": m * (rows * s + 16) + 4 * n * vectors, "flops": 0}
    if op == "route":
        t, e, k = case["t"], case["e"], case["k"]
        # logits in; experts, shares, places and order out; backward the shares' gradients in and the logits' out
        moved = t * (e * s + k * 16) + 4 * (e + 1)
        return {"bytes": moved + (t * (e * s + k * 4) if case["backward"] else 0), "flops": 0}
    if op in ("dispatch", "combine"):
        t, h, k = case["t"], case["h"], case["k"]
        rows = t * h * (1 + k * (1.0 - case["masked"]))
        if op == "dispatch":
            return {"bytes": rows * s + t * k * 4, "flops": 0}
        if case["backward"]:
            return {"bytes": (rows + t * h * k * (1.0 - case["masked"])) * s + t * k * 12, "flops": 0}
        return {"bytes": (rows + t * h * case["residual"]) * s + t * k * 8, "flops": 0}
    if op == "keep8":
        m, n = case["m"], case["n"]
        return {"bytes": m * n * (2 * s + 2) + 2 * m * ((n + 31) // 32), "flops": 0}
    m, n, k = case["m"], case["n"], case["k"]
    moved = (m * n + m * k + 2 * n * k) * s + m * (k + (k + 31) // 32)
    if case["act"] != "none":
        moved += m * (n + (n + 31) // 32)
    return {"bytes": moved + 4 * n * case["bias"], "flops": 4.0 * m * n * k}


# ------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt, op = TYPES[case["dtype"]], case["op"]
    pad = case.get("pad", 0)

    def normal(rows, cols, std=1.0, mean=0.0, pad=0):
        """[rows][cols] values; with pad the rows are pad elements further apart than cols."""
        t = torch.randn(rows, cols + pad, generator=g, device=DEV, dtype=torch.float32).mul_(std).add_(mean).to(dt)
        return t[:, :cols] if pad else t

    def vector(n, mean, std):
        return torch.randn(n, generator=g, device=DEV).mul_(std).add_(mean)

    def empty(rows, cols):
        return torch.empty(rows, cols, dtype=dt, device=DEV)

    s = dict(case)
    if op == "norm":
        m, n, post, pre, extras = (case[x] for x in ("m", "n", "post", "pre", "extras"))
        s["y"] = normal(m, n, 1.5, 0.1, pad) if post else None
        s["g"] = None if case["gate"] == "none" else normal(m, 1 if case["per_row"] else n, 1.0, 0.3, 0 if case["per_row"] else pad)
        s["res"] = normal(m, n, 2.0, 0.05, pad)
        s["w_post"] = vector(n, 1.0, 0.2) if post else None
        s["b_post"] = vector(n, 0.0, 0.1) if post and extras else None
        s["scale"] = vector(n, 0.5, 0.1) if post and extras else None
        s["w_pre"] = vector(n, 1.0, 0.2) if pre else None
        s["b_pre"] = vector(n, 0.0, 0.1) if pre and extras else None
        s["stats"] = torch.zeros(m, 4, device=DEV)
        if not case["backward"]:
            s["r"] = empty(m, n) if post else None
            s["h"] = empty(m, n) if pre else None
        else:
            r, _, stats = _plain_norm(s)
            s["r"] = (r if post else s["res"]) if pre else None
            s["stats"].copy_(stats)
            s["dr"] = normal(m, n, 1e-2, 0.0, pad) if extras or not pre else None
            s["dh"] = normal(m, n, 1e-2, 0.0, pad) if pre else None
            s["out"] = {"residual": empty(m, n)}
            if post:
                s["out"]["y"] = empty(m, n)
                s["out"]["w_post"] = torch.empty(n, device=DEV)
                if case["gate"] != "none":
                    s["out"]["gate"] = torch.empty_like(s["g"], memory_format=torch.contiguous_format)
                if extras:
                    s["out"]["b_post"], s["out"]["scale"] = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
            if pre:
                s["out"]["w_pre"] = torch.empty(n, device=DEV)
                if extras:
                    s["out"]["b_pre"] = torch.empty(n, device=DEV)
    elif op == "route":
        t, e, k = case["t"], case["e"], case["k"]
        s["logits"] = normal(t, e, 2.0)
        if case["masked"]:   # experts closed to a sample; now and then all of them
            closed = torch.rand(t, e, generator=g, device=DEV) < case["masked"]
            closed |= torch.rand(t, 1, generator=g, device=DEV) < 0.01
            s["logits"] = s["logits"].masked_fill(closed, -math.inf)
        s["d_probs"] = torch.randn(t, k, generator=g, device=DEV).mul_(1e-2) if case["backward"] else None
        s["ids"] = torch.empty(t, k, dtype=torch.int32, device=DEV)
        s["probs"] = torch.empty(t, k, device=DEV)
        s["slots"], s["order"] = torch.empty(t, k, dtype=torch.int32, device=DEV), torch.empty(t * k, dtype=torch.int32, device=DEV)
        s["offsets"] = torch.empty(e + 1, dtype=torch.int32, device=DEV)
        s["d_logits"] = empty(t, e) if case["backward"] else None
    elif op in ("dispatch", "combine"):
        t, h, k, e = (case[x] for x in "thke")
        # experts are chosen unevenly, as trained routers choose them
        lean = torch.randn(1, e, generator=g, device=DEV)
        pick = torch.argsort(torch.rand(t, e, generator=g, device=DEV).log().neg().log().neg() + lean, dim=1, descending=True)
        ids = pick[:, :k] if k <= e else torch.randint(e, (t, k), generator=g, device=DEV)
        if case["masked"]:
            ids = ids.masked_fill(torch.rand(t, k, generator=g, device=DEV) < case["masked"], -1)
        s["slots"], _, s["offsets"] = _plain_sort(ids, e)
        s["probs"] = torch.softmax(torch.randn(t, k, generator=g, device=DEV), 1)
        if op == "dispatch" and not case["backward"]:
            s["x"], s["out"] = normal(t, h, pad=pad), torch.zeros(t * k, h, dtype=dt, device=DEV)
        elif op == "dispatch":
            s["d_xs"], s["out"] = normal(t * k, h, 1e-2, pad=pad), empty(t, h)
        elif not case["backward"]:
            s["ys"], s["out"] = normal(t * k, h, pad=pad), empty(t, h)
            s["res"] = normal(t, h, pad=pad) if case["residual"] else None
        else:
            s["ys"], s["dy"] = normal(t * k, h, pad=pad), normal(t, h, 1e-2, pad=pad)
            s["out"], s["d_probs"] = torch.zeros(t * k, h, dtype=dt, device=DEV), torch.empty(t, k, device=DEV)
    elif op == "keep8":
        m, n = case["m"], case["n"]
        s["x"] = normal(m, n, pad=pad)
        s["q"] = torch.empty(m, n, dtype=torch.uint8, device=DEV)
        s["exps"] = torch.empty(m, (n + 31) // 32, dtype=torch.uint8, device=DEV)
        s["out"] = empty(m, n)
    else:
        m, n, k = case["m"], case["n"], case["k"]
        s["rng"] = torch.tensor([seed * 2654435761 + 12345, 7 * seed + 1], dtype=torch.int64, device=DEV)
        s["dy"] = normal(m, n, 1e-2, pad=pad)
        s["xq"], s["xe"] = _plain_pack(normal(m, k))
        s["zq"], s["ze"] = _plain_pack(normal(m, n)) if case["act"] != "none" else (None, None)
        lim = math.sqrt(6.0 / (n + k))   # Xavier-uniform, as the layers are initialised
        s["w"] = torch.rand(n, k, generator=g, device=DEV).mul_(2 * lim).sub_(lim).to(dt)
        s["dx"], s["dw"] = empty(m, k), empty(n, k)
        s["db"] = torch.empty(n, device=DEV) if case["bias"] else None
    if own:
        import dlrm_embeddings_dot_gb300 as dl
        s["dl"], size = dl, 0
        if op == "norm":
            s["norm_code"] = dl.DLRM_NORM_RMS if case["kind"] == "rms" else dl.DLRM_NORM_LAYER
            s["gate_code"] = {"none": dl.DLRM_GATE_NONE, "raw": dl.DLRM_GATE_NONE, "sigmoid": dl.DLRM_GATE_SIGMOID,
                              "silu": dl.DLRM_GATE_SILU}[case["gate"]]
            if case["backward"]:
                size = dl.dlrm_block_norm_bwd_workspace_size(s["res"])
        elif op == "route":
            size = dl.dlrm_expert_sort_workspace_size(s["ids"], case["e"])
        elif op == "grad8":
            s["act_code"] = {"none": dl.DLRM_ACT_NONE, "relu": dl.DLRM_ACT_RELU, "gelu": dl.DLRM_ACT_GELU,
                             "silu": dl.DLRM_ACT_SILU}[case["act"]]
            size = dl.dlrm_linear_bwd8_workspace_size(s["dy"], s["xq"], s["w"], act=s["act_code"], p=case["p"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV) if size else None
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _row_stats(v, kind):
    mean = v.mean(1) if kind == "layer" else torch.zeros(v.shape[0], device=DEV)
    c = v - mean[:, None]
    return mean, 1 / torch.sqrt((c * c).mean(1) + EPS)


def _gate(g, kind):
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-g))
    return g / (1 + torch.exp(-g)) if kind == "silu" else g


def _gate_slope(g, kind):
    if kind == "raw":
        return torch.ones_like(g)
    v = 1 / (1 + torch.exp(-g))
    return v * (1 - v) if kind == "sigmoid" else v * (1 + g * (1 - v))


def _plain_norm(s):
    dt, kind = s["res"].dtype, s["kind"]
    r, h, stats = s["res"].float(), None, torch.zeros(s["m"], 4, device=DEV)
    if s["post"]:
        y = s["y"].float()
        stats[:, 0], stats[:, 1] = _row_stats(y, kind)
        u = (y - stats[:, :1]) * stats[:, 1:2] * s["w_post"]
        if s["b_post"] is not None:
            u = u + s["b_post"]
        if s["g"] is not None:
            u = u * _gate(s["g"].float(), s["gate"])
        if s["scale"] is not None:
            u = u * s["scale"]
        r = r + u
    if s["pre"]:
        stats[:, 2], stats[:, 3] = _row_stats(r, kind)
        h = (r - stats[:, 2:3]) * stats[:, 3:] * s["w_pre"]
        h = (h if s["b_pre"] is None else h + s["b_pre"]).to(dt)
    return r.to(dt), h, stats


def _plain_norm_fwd(s):
    r, h, stats = _plain_norm(s)
    return {k: v for k, v in (("r", r if s["post"] else None), ("h", h), ("stats", stats)) if v is not None}


def _norm_grad(d, x, rstd, layer):
    """Gradient through x = (v - mean) rstd."""
    d = d - x * (d * x).mean(1, keepdim=True) - (d.mean(1, keepdim=True) if layer else 0)
    return d * rstd


def _norm_bwd(s, wide):
    """The backward's formulas in the type that `wide` takes the inputs to."""
    layer, out = s["kind"] == "layer", {}
    st = wide(s["stats"])
    dr = 0 if s["dr"] is None else wide(s["dr"])
    if s["pre"]:
        rn, dh = (wide(s["r"]) - st[:, 2:3]) * st[:, 3:], wide(s["dh"])
        dr = dr + _norm_grad(dh * wide(s["w_pre"]), rn, st[:, 3:], layer)
        out["w_pre"] = (dh * rn).sum(0)
        if s["extras"]:
            out["b_pre"] = dh.sum(0)
    out["residual"] = dr
    if s["post"]:
        yn = (wide(s["y"]) - st[:, :1]) * st[:, 1:2]
        u = yn * wide(s["w_post"]) + (0 if s["b_post"] is None else wide(s["b_post"]))
        gate = 1 if s["g"] is None else _gate(wide(s["g"]), s["gate"])
        scale = 1 if s["scale"] is None else wide(s["scale"])
        du = dr * gate * scale
        out["y"] = _norm_grad(du * wide(s["w_post"]), yn, st[:, 1:2], layer)
        out["w_post"] = (du * yn).sum(0)
        if s["extras"]:
            out["b_post"], out["scale"] = du.sum(0), (dr * gate * u).sum(0)
        if s["g"] is not None:
            dg = dr * scale * u
            if s["per_row"]:
                dg = dg.sum(1, keepdim=True)
            out["gate"] = dg * _gate_slope(wide(s["g"]), s["gate"])
    return out


def _plain_norm_bwd(s):
    got = _norm_bwd(s, torch.Tensor.float)
    return {k: got[k].to(v.dtype) for k, v in s["out"].items()}


def _plain_sort(ids, e):
    """(places [T][k], order, offsets): choices by expert, then by position; those without expert behind, -1."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < e), flat, e)
    order = torch.argsort(key, stable=True)
    offsets = torch.zeros(e + 2, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(torch.zeros(e + 1, dtype=torch.int64, device=DEV).scatter_add_(0, key, torch.ones_like(key)), 0)
    place = torch.arange(n, device=DEV)
    slots = torch.empty_like(order).scatter_(0, order, place)
    slots = torch.where(key < e, slots, -1)
    order = torch.where(place < offsets[e], order, -1)
    return slots.view(ids.shape).to(torch.int32), order.to(torch.int32), offsets[:e + 1].to(torch.int32)


def _plain_route(s):
    k, logits = s["k"], s["logits"].float()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    is_open = top != -math.inf
    ids = torch.where(is_open, ids, -1)
    probs = torch.where(is_open, torch.exp(top - torch.where(is_open[:, :1], top[:, :1], 0.0)), 0.0)
    probs = probs / torch.where(is_open[:, :1], probs.sum(1, keepdim=True), 1.0)
    slots, order, offsets = _plain_sort(ids, s["e"])
    out = {"ids": ids.to(torch.int32), "probs": probs, "slots": slots, "order": order, "offsets": offsets}
    if s["backward"]:
        d = probs * (s["d_probs"] - (s["d_probs"] * probs).sum(1, keepdim=True))
        grad = torch.zeros(s["t"], s["e"] + 1, device=DEV).scatter_(1, torch.where(is_open, ids, s["e"]), torch.where(is_open, d, 0.0))
        out["d_logits"] = grad[:, :s["e"]].to(s["logits"].dtype)
    return out


def _placed(rows, slots, wide):
    """rows[slots] as [T][k][H], zeros where there is no place."""
    at = slots.long()
    return torch.where(at[:, :, None] >= 0, wide(rows[at.clamp(min=0)]), 0.0)


def _to_places(values, slots, like):
    """values [T][k][H] at their places; the other rows zero, as they were."""
    t, k, h = values.shape
    out = torch.zeros(t * k + 1, h, dtype=like.dtype, device=DEV)
    at = slots.reshape(-1).long()
    out[torch.where(at >= 0, at, t * k)] = values.reshape(t * k, h).to(like.dtype)
    return out[:t * k]


def _plain_experts(s):
    slots, t, k, h = s["slots"], s["t"], s["k"], s["h"]
    if s["op"] == "dispatch":
        if not s["backward"]:
            return {"xs": _to_places(s["x"].unsqueeze(1).expand(t, k, h), slots, s["x"])}
        return {"dx": _placed(s["d_xs"], slots, torch.Tensor.float).sum(1).to(s["d_xs"].dtype)}
    ys, probs = _placed(s["ys"], slots, torch.Tensor.float), s["probs"]
    if not s["backward"]:
        y = (ys * probs[:, :, None]).sum(1)
        if s["res"] is not None:
            y = y + s["res"].float()
        return {"y": y.to(s["ys"].dtype)}
    dy = s["dy"].float()[:, None]
    return {"dys": _to_places(dy * probs[:, :, None], slots, s["ys"]), "d_probs": (ys * dy).sum(2)}


def _plain_pack(x):
    """(8-bit floats [M][N] as bytes, powers of two [M][N / 32] as bytes): blocks of 32 columns share the least power of
    two that takes their largest value to 448 or less; values are rounded to 4 significant bits, 2^-9 the least."""
    m, n = x.shape
    blocks = (n + 31) // 32
    v = torch.zeros(m, blocks * 32, device=DEV)
    v[:, :n] = x.float()
    v = v.view(m, blocks, 32)
    frac, exp = torch.frexp(v.abs().amax(2))        # largest = frac 2^exp, frac in [0.5, 1)
    e = (exp - 9 + (frac > 0.875).int() + 127).clamp(min=0)
    e = torch.where(frac == 0, 0, e)
    v = torch.ldexp(torch.ldexp(v, ((127 - e) // 2)[:, :, None]), ((128 - e) // 2)[:, :, None])
    _, exp = torch.frexp(v)
    step = torch.clamp(exp - 4, min=-9)             # of the 4 bits, or of the smallest values
    i = torch.round(torch.ldexp(v, -step))          # up to 16 in size
    size = i.abs().int()
    up = (size == 16).int()                         # rounded up to the next power of two
    size, step = torch.where(up > 0, 8, size), step + up
    bits = torch.where(size < 8, size, (step + 10) * 8 + size - 8) + (v < 0).int() * 128
    return bits.view(m, blocks * 32)[:, :n].to(torch.uint8).contiguous(), e.to(torch.uint8)


def _plain_unpack(q, exps, dtype, wide=torch.Tensor.float):
    b = q.int()
    mant, ex = b & 7, b >> 3 & 15
    v = torch.where(ex > 0, wide(mant + 8) * torch.exp2(wide(ex - 10)), wide(mant) * 2.0**-9) * torch.where(b > 127, -1.0, 1.0)
    e = exps.int().repeat_interleave(32, 1)[:, :q.shape[1]] - 127
    v = v * torch.exp2(wide(e // 2)) * torch.exp2(wide((e + 1) // 2))
    return v.clamp(-LARGEST[dtype], LARGEST[dtype])


def _plain_keep8(s):
    q, exps = _plain_pack(s["x"])
    return {"y": _plain_unpack(q, exps, s["dtype"]).to(s["x"].dtype)}


def _keep_scale(rng, m, n, p):
    """[m][n] fp32: 0 where the element is dropped, 1/(1-p) where it is kept.  Philox4x32-10 (Salmon et al., SC 2011)
    keyed by rng[0] with counter (column / 8, row, rng[1]); eight 16-bit numbers an output, one a column."""
    low = 0xFFFFFFFF
    groups = (n + 7) // 8
    c0 = torch.arange(groups, device=DEV).repeat(m)
    c1 = torch.arange(m, device=DEV).repeat_interleave(groups)
    c2, c3 = (rng[1] & low).expand(m * groups), ((rng[1] >> 32) & low).expand(m * groups)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((c0, c1, c2, c3), dim=1)
    u = torch.stack((words & 0xFFFF, words >> 16), dim=2).reshape(m, groups * 8)[:, :n]
    thr = math.floor(p * 65536 + 0.5)
    return torch.where(u >= thr, 65536.0 / (65536 - thr), 0.0)


def _act_grad(z, act):
    if act == "relu":
        return torch.where(z <= 0, 0.0, 1.0)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    v = 1 / (1 + torch.exp(-z))
    return v * (1 + z * (1 - v))


def _plain_grad8(s):
    dt, name = s["dy"].dtype, s["dtype"]
    dz = s["dy"].float()
    if s["p"] > 0:
        dz = dz * _keep_scale(s["rng"], s["m"], s["n"], s["p"])
    if s["act"] != "none":
        dz = dz * _act_grad(_plain_unpack(s["zq"], s["ze"], name), s["act"])
    out = {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ _plain_unpack(s["xq"], s["xe"], name)).to(dt)}
    if s["bias"]:
        out["db"] = dz.sum(0)
    return out


def run(s):
    op = s["op"]
    if not own:
        if op == "norm":
            return _plain_norm_bwd(s) if s["backward"] else _plain_norm_fwd(s)
        return {"route": _plain_route, "dispatch": _plain_experts, "combine": _plain_experts, "keep8": _plain_keep8,
                "grad8": _plain_grad8}[op](s)
    dl = s["dl"]
    if op == "norm" and not s["backward"]:
        dl.dlrm_block_norm_fwd(s["y"], s["g"], s["res"], s["w_post"], s["b_post"], s["scale"], s["w_pre"], s["b_pre"], s["r"],
                               s["h"], s["stats"], norm=s["norm_code"], gate_act=s["gate_code"], eps=EPS)
        return {k: s[k] for k in ("r", "h", "stats") if s[k] is not None}
    if op == "norm":
        o = s["out"]
        dl.dlrm_block_norm_bwd(s["dr"], s["dh"], s["y"], s["g"], s["r"], s["stats"], s["w_post"], s["b_post"], s["scale"],
                               s["w_pre"], o.get("y"), o.get("gate"), o["residual"], o.get("w_post"), o.get("b_post"),
                               o.get("scale"), o.get("w_pre"), o.get("b_pre"), norm=s["norm_code"], gate_act=s["gate_code"],
                               workspace=s["ws"])
        return o
    if op == "route":
        dl.dlrm_route_fwd(s["logits"], s["ids"], s["probs"])
        dl.dlrm_expert_sort(s["ids"], s["e"], s["offsets"], s["slots"], s["order"], workspace=s["ws"])
        out = {k: s[k] for k in ("ids", "probs", "slots", "order", "offsets")}
        if s["backward"]:
            dl.dlrm_route_bwd(s["d_probs"], s["ids"], s["probs"], s["d_logits"])
            out["d_logits"] = s["d_logits"]
        return out
    if op == "dispatch":
        if s["backward"]:
            dl.dlrm_dispatch_bwd(s["d_xs"], s["slots"], s["out"])
            return {"dx": s["out"]}
        dl.dlrm_dispatch_fwd(s["x"], s["slots"], s["out"])
        return {"xs": s["out"]}
    if op == "combine":
        if s["backward"]:
            dl.dlrm_combine_bwd(s["dy"], s["ys"], s["slots"], s["probs"], s["out"], s["d_probs"])
            return {"dys": s["out"], "d_probs": s["d_probs"]}
        dl.dlrm_combine_fwd(s["ys"], s["slots"], s["probs"], s["res"], s["out"])
        return {"y": s["out"]}
    if op == "keep8":
        dl.dlrm_pack8(s["x"], s["q"], s["exps"])
        dl.dlrm_unpack8(s["q"], s["exps"], s["out"])
        return {"y": s["out"]}
    dl.dlrm_linear_bwd8(s["dy"], s["xq"], s["xe"], s["w"], s["zq"], s["ze"], s["dx"], s["dw"], s["db"], act=s["act_code"],
                        p=s["p"], rng=s["rng"], workspace=s["ws"])
    return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]} if s["bias"] else {"dx": s["dx"], "dw": s["dw"]}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _exact_norm(s):
    kind = s["kind"]

    def normed(v):
        mean = v.sum(1, keepdim=True) / v.shape[1] if kind == "layer" else torch.zeros_like(v[:, :1])
        rstd = (((v - mean) ** 2).sum(1, keepdim=True) / v.shape[1] + EPS) ** -0.5
        return mean, rstd, (v - mean) * rstd

    r, out, zero = s["res"].double(), {}, torch.zeros(s["m"], 1, dtype=torch.float64, device=DEV)
    stats = [zero, zero, zero, zero]
    if s["post"]:
        stats[0], stats[1], u = normed(s["y"].double())
        u = u * s["w_post"].double() + (0 if s["b_post"] is None else s["b_post"].double())
        if s["g"] is not None:
            g = s["g"].double()
            u = u * {"raw": g, "sigmoid": torch.sigmoid(g), "silu": g * torch.sigmoid(g)}[s["gate"]]
        r = r + u * (1 if s["scale"] is None else s["scale"].double())
        out["r"] = r
    if s["pre"]:
        stats[2], stats[3], h = normed(r)
        out["h"] = h * s["w_pre"].double() + (0 if s["b_pre"] is None else s["b_pre"].double())
    out["stats"] = torch.cat(stats, 1)
    return out


def _exact_norm_bwd(s):
    """By way of autograd: the forward in 64 bits with the kept statistics' values, the norms' own gradients through the
    identities for a row of mean 0 and mean square 1."""
    st, layer, n = s["stats"].double(), s["kind"] == "layer", s["n"]
    dr = torch.zeros(s["m"], n, dtype=torch.float64, device=DEV) if s["dr"] is None else s["dr"].double()
    out = {}

    def back(d, v, mean, rstd):
        x = (v - mean) * rstd
        g = d - x * ((d * x).sum(1, keepdim=True) / n)
        return rstd * (g - d.sum(1, keepdim=True) / n if layer else g), x

    if s["pre"]:
        dh = s["dh"].double()
        more, x = back(dh * s["w_pre"].double(), s["r"].double(), st[:, 2:3], st[:, 3:])
        dr = dr + more
        out["w_pre"], out["b_pre"] = torch.einsum("mn,mn->n", dh, x), dh.sum(0)
    out["residual"] = dr
    if s["post"]:
        leaf = None if s["g"] is None else s["g"].double().requires_grad_()
        gate = torch.ones(1, 1, dtype=torch.float64, device=DEV)
        if leaf is not None:
            gate = {"raw": lambda v: v, "sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu}[s["gate"]](leaf)
        one = torch.ones(n, dtype=torch.float64, device=DEV)
        scale = one if s["scale"] is None else s["scale"].double()
        shift = 0 * one if s["b_post"] is None else s["b_post"].double()
        w = s["w_post"].double()
        x = (s["y"].double() - st[:, :1]) * st[:, 1:2]
        u = x * w + shift
        if leaf is not None:
            (gate * (dr * scale * u)).sum().backward()
            out["gate"] = leaf.grad
            gate = gate.detach()
        a = dr * gate
        out["y"], _ = back(a * scale * w, s["y"].double(), st[:, :1], st[:, 1:2])
        out["w_post"], out["b_post"], out["scale"] = (a * scale * x).sum(0), (a * scale).sum(0), (a * u).sum(0)
    return {k: out[k] for k in s["out"]}


def _exact_unpack(q, exps, dtype):
    """The table of the format's 256 values, times the blocks' powers of two."""
    table = [0.0] * 256
    for b in range(256):
        ex, mant = b >> 3 & 15, b & 7
        v = (1 + mant / 8) * 2.0 ** (ex - 7) if ex else mant / 8 * 2.0**-6
        table[b] = math.nan if b & 127 == 127 else -v if b & 128 else v
    v = torch.tensor(table, dtype=torch.float64, device=DEV)[q.long()]
    blocks = torch.tensor([2.0 ** (b - 127) for b in range(256)], dtype=torch.float64, device=DEV)[exps.long()]
    v = v * blocks.repeat_interleave(32, 1)[:, :q.shape[1]]
    return torch.minimum(torch.maximum(v, torch.full_like(v, -LARGEST[dtype])), torch.full_like(v, LARGEST[dtype]))


def _exact_pack(x):
    """Bytes by search: the nearest of the format's values, the even one of two as near."""
    m, n = x.shape
    v = torch.zeros(m, -(-n // 32) * 32, dtype=torch.float64, device=DEV)
    v[:, :n] = x.double()
    v = v.view(m, -1, 32)
    big = v.abs().amax(2)
    e = torch.where(big > 0, torch.ceil(torch.log2(big / 448.0)), -127.0).clamp(min=-127)
    e = torch.where(big > 448.0 * torch.exp2(e), e + 1, torch.where((big <= 224.0 * torch.exp2(e)) & (e > -127), e - 1, e))
    sizes = torch.tensor([(1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 7) if b >> 3 else (b & 7) / 8 * 2.0**-6 for b in range(127)],
                         dtype=torch.float64, device=DEV)
    middle = (sizes[1:] + sizes[:-1]) / 2
    a = (v.abs() / torch.exp2(e)[:, :, None]).reshape(m, -1)
    below, above = torch.searchsorted(middle, a), torch.searchsorted(middle, a, right=True)
    b = torch.where(below == above, below, torch.where(below % 2 == 0, below, above))
    b = b + (v.reshape(m, -1) < 0) * 128
    return b[:, :n].to(torch.uint8), (e + 127).to(torch.uint8)


def _exact_scale(rng, m, n, p):
    seed, offset = (int(v) % 2**64 for v in rng.tolist())
    u32, m32 = np.uint64(32), np.uint64(2**32 - 1)
    groups = -(-n // 8)
    w = [np.tile(np.arange(groups, dtype=np.uint64), (m, 1)), np.repeat(np.arange(m, dtype=np.uint64)[:, None], groups, 1),
         np.full((m, groups), offset % 2**32, np.uint64), np.full((m, groups), offset >> 32, np.uint64)]
    key = [seed % 2**32, seed >> 32]
    for r in range(10):
        p0, p1 = w[0] * np.uint64(0xD2511F53), w[2] * np.uint64(0xCD9E8D57)
        w = [(p1 >> u32) ^ w[1] ^ np.uint64(key[0]), p1 & m32, (p0 >> u32) ^ w[3] ^ np.uint64(key[1]), p0 & m32]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    u = np.empty((m, groups, 8), np.uint16)
    for j in range(4):
        u[:, :, 2 * j] = (w[j] & np.uint64(0xFFFF)).astype(np.uint16)
        u[:, :, 2 * j + 1] = (w[j] >> np.uint64(16)).astype(np.uint16)
    thr = int(math.floor(p * 65536 + 0.5))
    kept = torch.from_numpy(u.reshape(m, groups * 8)[:, :n] >= thr).to(DEV)
    return kept.double() * (65536.0 / (65536 - thr))


def _exact_slope(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm_bwd(s) if case["backward"] else _exact_norm(s)
    if op == "route":
        out = {"ids": None, "probs": None, "slots": None, "order": None, "offsets": None}
        logits = s["logits"].double()
        ids = torch.argsort(-logits, dim=1, stable=True)[:, :case["k"]]
        top = torch.gather(logits, 1, ids)
        probs = torch.nan_to_num(torch.softmax(top, dim=1), nan=0.0)   # rows without an open expert
        out["probs"] = probs
        if case["backward"]:
            d = s["d_probs"].double()
            d = probs * (d - (d * probs).sum(1, keepdim=True))
            out["d_logits"] = torch.zeros_like(logits).scatter_(1, ids, d)
        return out
    if op in ("dispatch", "combine"):
        at = s["slots"].reshape(-1).long()
        here = torch.nonzero(at >= 0)[:, 0]
        at, token = at[here], here // case["k"]
        t, h, k = case["t"], case["h"], case["k"]
        if op == "dispatch" and not case["backward"]:
            out = torch.zeros(t * k, h, dtype=torch.float64, device=DEV)
            out[at] = s["x"].double()[token]
            return {"xs": out}
        if op == "dispatch":
            return {"dx": torch.zeros(t, h, dtype=torch.float64, device=DEV).index_add_(0, token, s["d_xs"].double()[at])}
        probs = s["probs"].double().reshape(-1)[here][:, None]
        if not case["backward"]:
            y = torch.zeros(t, h, dtype=torch.float64, device=DEV) if s["res"] is None else s["res"].double().clone()
            return {"y": y.index_add_(0, token, s["ys"].double()[at] * probs)}
        dy = s["dy"].double()[token]
        out = torch.zeros(t * k, h, dtype=torch.float64, device=DEV)
        out[at] = dy * probs
        d = torch.zeros(t * k, dtype=torch.float64, device=DEV)
        d[here] = torch.einsum("ih,ih->i", s["ys"].double()[at], dy)
        return {"dys": out, "d_probs": d.view(t, k)}
    if op == "keep8":
        return {"y": _exact_unpack(*_exact_pack(s["x"]), case["dtype"])}
    dz = s["dy"].double()
    if case["p"] > 0:
        dz = dz * _exact_scale(s["rng"], case["m"], case["n"], case["p"])
    if case["act"] != "none":
        dz = dz * _exact_slope(_exact_unpack(s["zq"], s["ze"], case["dtype"]), case["act"])
    out = {"dx": dz @ s["w"].double(), "dw": dz.t() @ _exact_unpack(s["xq"], s["xe"], case["dtype"])}
    if case["bias"]:
        out["db"] = dz.sum(0)
    return out
