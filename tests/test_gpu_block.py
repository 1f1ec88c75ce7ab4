"""The residual blocks' operators on the GPU (include/dlrm_block.h) against plain 64-bit forms
(``block_ref``, which also derives the error bounds)."""

import pytest
import torch

import block_ref as ref
import dense_ref as dref
from gpu_util import dev

pytestmark = pytest.mark.gpu

DTYPES = ["f32", "f16", "bf16"]
INF, NAN = float("inf"), float("nan")
LARGEST = {"f32": 3.3895313892515355e38, "f16": 65504.0, "bf16": 3.3895313892515355e38}


def _rand(g, *shape, std=1.0, mean=0.0, dtype="f32", pad=0, lead=0):
    """Normal values on the device; pad: extra columns between rows; lead: elements before the first."""
    t = torch.randn(*shape[:-1], shape[-1] + pad + lead, generator=g, dtype=torch.float64) * std + mean
    return t.to(dref.TYPES[dtype]).to(dev())[..., lead:lead + shape[-1]]


def _empty(M, N, dtype, pad=0, lead=0):
    """Output with guard columns that must stay as they are."""
    return torch.full((M, lead + N + pad), 7.0, dtype=dref.TYPES[dtype], device=dev())[:, lead:lead + N]


def _guard_ok(t):
    if t._base is None:
        return True
    b, lead = t._base, t.storage_offset()
    return bool((b[:, :lead] == 7.0).all()) and bool((b[:, lead + t.shape[1]:] == 7.0).all())


def _ws(n):
    return torch.empty(n, dtype=torch.uint8, device=dev()) if n else None


def _d(t):
    return None if t is None else t.double().cpu()


# ------------------------------------------------------------------------------------------- norms
SHAPES = [(1, 1, 0, 0), (1, 8, 0, 0), (3, 7, 0, 0), (2, 33, 3, 1), (5, 256, 0, 0), (2, 257, 0, 0), (37, 480, 8, 0),
          (300, 1024, 0, 0), (3, 1032, 8, 0), (9, 2048, 0, 1), (2, 2500, 0, 0), (4, 4100, 0, 0), (3, 8192, 0, 0),
          (2, 8191, 0, 0), (2600, 96, 0, 0), (700, 515, 0, 0), (5000, 16, 0, 0), (333, 32, 8, 0), (77, 64, 0, 1),
          (65, 128, 8, 0), (513, 128, 0, 0), (19, 200, 0, 0), (9, 1999, 1, 0),
          (2000, 700, 0, 0), (1300, 1200, 8, 0), (900, 1501, 0, 0), (700, 1720, 0, 1), (600, 2304, 0, 0), (500, 2903, 0, 0),
          (400, 4800, 0, 0), (333, 6001, 0, 0)]
OPTIONS = [   # layer, gate, per row, block, next norm, vectors, residual
    (False, None, False, True, True, False, True), (False, "silu", False, True, True, True, True),
    (True, "sigmoid", True, True, True, True, True), (True, "raw", False, True, False, True, False),
    (False, None, False, False, True, True, True), (True, "silu", True, True, False, False, True)]


def _norm_case(seed, M, N, pad, lead, dtype, option):
    layer, gate, per_row, post, pre, vectors, residual = option
    g = torch.Generator().manual_seed(seed)
    kw = dict(dtype=dtype, pad=pad, lead=lead)
    v = lambda mean: _rand(g, N, std=0.3, mean=mean)
    return dict(
        y=_rand(g, M, N, std=1.5, mean=0.2, **kw) if post else None,
        gate=None if gate is None else _rand(g, M, 1 if per_row else N, mean=0.3, **kw),
        residual=_rand(g, M, N, std=2.0, mean=-0.1, **kw) if residual else None,
        w_post=v(1.0) if post else None, b_post=v(0.0) if post and vectors else None,
        scale=v(0.5) if post and vectors else None, w_pre=v(1.0) if pre else None, b_pre=v(0.0) if pre and vectors else None)


def _codes(dl, option):
    norm = dl.DLRM_NORM_LAYER if option[0] else dl.DLRM_NORM_RMS
    return dict(norm=norm, gate_act=ref.GATES[option[1] or "raw"])


def _forward(dl, a, option, M, N, dtype, pad=0, lead=0, eps=1e-5, stats=True):
    r = _empty(M, N, dtype, pad, lead) if option[3] else None
    h = _empty(M, N, dtype, pad, lead) if option[4] else None
    st = torch.full((M, 4), 7.0, device=dev()) if stats else None
    dl.dlrm_block_norm_fwd(a["y"], a["gate"], a["residual"], a["w_post"], a["b_post"], a["scale"], a["w_pre"], a["b_pre"], r, h,
                           st, eps=eps, **_codes(dl, option))
    return r, h, st


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("option", OPTIONS)
@pytest.mark.parametrize("M,N,pad,lead", SHAPES)
def test_norm_forward(cuda_lib, dtype, option, M, N, pad, lead):
    a = _norm_case(M * N, M, N, pad, lead, dtype, option)
    r, h, st = _forward(cuda_lib, a, option, M, N, dtype, pad, lead)
    want = ref.forward(*(_d(a[k]) for k in ("y", "gate", "residual", "w_post", "b_post", "scale", "w_pre", "b_pre")), option[0],
                       option[1] or "raw", 1e-5, option[4])
    for name, got in (("r", r), ("h", h)):
        if got is not None:
            dref.assert_close(got, *want[name], dtype, name)
            assert _guard_ok(got)
    zero = torch.zeros(M, 1, dtype=torch.float64)
    for name, at, on in (("y_stats", 0, option[3]), ("r_stats", 2, option[4])):
        m, s = want[name] if on else (zero, zero)
        # statistics to 32 bits: the mean by its sum's bound, 1 / sqrt by the norm's relative bound
        v = a["y"] if at == 0 else None
        size = _d(v).abs().mean(1, keepdim=True) if v is not None else (_d(r if r is not None else a["residual"])).abs().mean(1, keepdim=True)
        assert ((_d(st)[:, at:at + 1] - m).abs() <= ((N + 16) * ref.SUM + (0.0 if at == 0 else 2.0**-8)) * size + 1e-30).all()
        assert ((_d(st)[:, at + 1:at + 2] - s).abs() <= ((N + 64) * ref.SUM + (0.0 if at == 0 else 2.0**-8)) * s * (1 + size * s)**2 + 1e-30).all()
    again = _forward(cuda_lib, a, option, M, N, dtype, pad, lead, stats=False)
    assert all(torch.equal(x, y) for x, y in zip((r, h), again) if x is not None)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("option", OPTIONS)
@pytest.mark.parametrize("M,N,pad,lead", SHAPES)
@pytest.mark.parametrize("paths", ["both", "h"])
def test_norm_backward(cuda_lib, dtype, option, M, N, pad, lead, paths):
    layer, gate, per_row, post, pre, vectors, residual = option
    if paths == "h" and not pre:
        pytest.skip("the gradient of r is all there is")
    a = _norm_case(M * N + 1, M, N, pad, lead, dtype, option)
    r, h, st = _forward(cuda_lib, a, option, M, N, dtype, pad, lead)
    r = (r if post else a["residual"]) if pre else None
    g = torch.Generator().manual_seed(7)
    gr = _rand(g, M, N, std=0.1, dtype=dtype, pad=pad, lead=lead) if paths == "both" else None
    gh = _rand(g, M, N, std=0.1, dtype=dtype, pad=pad, lead=lead) if pre else None
    out = {"residual": _empty(M, N, dtype, pad, lead)}
    vec = lambda: torch.full((N,), 7.0, device=dev())
    if post:
        out.update(y=_empty(M, N, dtype, pad, lead), w_post=vec(), b_post=vec(), scale=vec())
        if gate:
            out["gate"] = _empty(M, 1 if per_row else N, dtype, pad, lead)
    if pre:
        out.update(w_pre=vec(), b_pre=vec())
    ws = _ws(cuda_lib.dlrm_block_norm_bwd_workspace_size(gh if pre else gr))

    def run(o, ws):
        cuda_lib.dlrm_block_norm_bwd(gr, gh, a["y"], a["gate"], r, st, a["w_post"], a["b_post"], a["scale"], a["w_pre"],
                                     *(o.get(k) for k in ("y", "gate", "residual", "w_post", "b_post", "scale", "w_pre", "b_pre")),
                                     workspace=ws, **_codes(cuda_lib, option))

    run(out, ws)
    want = ref.backward(*(_d(t) for t in (gr, gh, a["y"], a["gate"], r, st, a["w_post"], a["b_post"], a["scale"], a["w_pre"])),
                        layer, gate or "raw")
    for k, got in out.items():
        dref.assert_close(got, *want[k], "f32" if got.dim() == 1 else dtype, k)
        assert got.dim() == 1 or _guard_ok(got)
    if M * N > 10000 or dtype != "f32":
        return
    for k in out:                    # each output alone, the same bits; the vectors' need the workspace
        alone = {k: torch.full_like(out[k], 3.0)}
        run(alone, ws if out[k].dim() == 1 else None)
        assert torch.equal(alone[k], out[k]), k


@pytest.mark.parametrize("N", [300, 515, 700, 1024, 1200, 1500, 1720])
def test_norm_backward_of_rows_that_share_a_block(cuda_lib, N):
    """Rows of one block go their own pace, with sums of one value and of two: every row right, every run the same."""
    M, option = 6000, OPTIONS[2]
    a = _norm_case(5, M, N, 0, 0, "f32", option)
    r, h, st = _forward(cuda_lib, a, option, M, N, "f32")
    g = torch.Generator().manual_seed(6)
    gh = _rand(g, M, N, std=0.1)
    want = ref.backward(None, *(_d(t) for t in (gh, a["y"], a["gate"], r, st, a["w_post"], a["b_post"], a["scale"], a["w_pre"])),
                        True, "sigmoid")
    first = None
    for _ in range(6):
        out = {"y": torch.empty_like(r), "gate": torch.empty_like(a["gate"]), "residual": torch.empty_like(r)}
        cuda_lib.dlrm_block_norm_bwd(None, gh, a["y"], a["gate"], r, st, a["w_post"], a["b_post"], a["scale"], a["w_pre"],
                                     *out.values(), *[None] * 5, **_codes(cuda_lib, option))
        first = first or out
        for k in out:
            dref.assert_close(out[k], *want[k], "f32", k)
            assert torch.equal(out[k], first[k])


@pytest.mark.parametrize("N", [16, 40, 100])
def test_norm_gradient_of_infinite_gates(cuda_lib, N):
    """Gates of infinity by row and gradients of 1: the bias's gradient is infinite, also where the last rows
    are fewer than a warp's."""
    M = 20001
    y, ones = torch.randn(M, N, device=dev()), torch.ones(M, N, device=dev())
    gate = torch.full((M, 1), INF, device=dev())
    st = torch.zeros(M, 4, device=dev())
    gb = torch.zeros(N, device=dev())
    ws = torch.empty(cuda_lib.dlrm_block_norm_bwd_workspace_size(y), dtype=torch.uint8, device=dev())
    cuda_lib.dlrm_block_norm_bwd(ones, None, y, gate, None, st, None, None, None, None, None, None, None, None, gb, None, None,
                                 None, workspace=ws)
    assert torch.equal(gb, torch.full_like(gb, INF))


def test_norm_rows_of_zeros_constants_and_numbers_that_are_none(cuda_lib):
    """A row of zeros is zeros (eps > 0), a constant row of LAYER its bias, infinities and NaN stay in their rows."""
    for layer in (False, True):
        x = torch.randn(6, 40, device=dev())
        x[1], x[2], x[3, 5], x[4, 7] = 0.0, 3.0, INF, NAN
        h, b = torch.empty_like(x), torch.randn(40, device=dev())
        cuda_lib.dlrm_block_norm_fwd(None, None, x, None, None, None, None, b, None, h, norm=int(layer))
        assert torch.equal(h[1], b) and (torch.equal(h[2], b) if layer else torch.allclose(h[2], 1 + b, atol=1e-5))
        assert h[[0, 5]].isfinite().all() and h[3:5].isnan().any(1).all() and h[4].isnan().all()
        cuda_lib.dlrm_block_norm_fwd(None, None, x, None, None, None, None, b, None, h, norm=int(layer), eps=0.0)
        assert h[1].isnan().all() and h[0].isfinite().all()


def test_norm_without_rows(cuda_lib):
    x = torch.empty(0, 24, device=dev())
    cuda_lib.dlrm_block_norm_fwd(x, None, x, None, None, None, None, None, x.clone(), x.clone())
    v = [torch.full((24,), 7.0, device=dev()) for _ in range(5)]
    cuda_lib.dlrm_block_norm_bwd(x, x, x, None, x, torch.empty(0, 4, device=dev()), None, None, None, None, None, None, None, *v)
    assert all((t == 0).all() for t in v)


def test_norm_of_values_far_from_their_spread(cuda_lib):
    """LAYER of 1000 + small: two passes keep the spread's digits (one pass of squares has none left)."""
    g = torch.Generator().manual_seed(2)
    x = _rand(g, 20, 700, std=0.05, mean=1000.0)
    h = torch.empty_like(x)
    cuda_lib.dlrm_block_norm_fwd(None, None, x, None, None, None, None, None, None, h, norm=cuda_lib.DLRM_NORM_LAYER)
    want = ref.forward(None, None, _d(x), None, None, None, None, None, True, "raw", 1e-6)["h"]
    dref.assert_close(h, *want, "f32")
    # the mean's rounding is the same for a row: below 2^-22 of 1000 over the spread
    assert float((_d(h) - want[0]).abs().max()) < 8 * 1000 * 2.0**-24 / 0.05


def test_norm_gradient_against_differences(cuda_lib):
    """Central differences of the kernel's forward in fp32 along random directions, h = 2^-6: truncation
    h^2 times the third derivative (some ten), rounding 2^-16 of the sums' sizes."""
    option = OPTIONS[2]
    M, N, eps = 12, 72, 1e-3
    a = _norm_case(3, M, N, 0, 0, "f32", option)
    g = torch.Generator().manual_seed(4)
    cr, ch = _rand(g, M, N, std=0.1), _rand(g, M, N, std=0.1)

    def loss(v):
        r, h, _ = _forward(cuda_lib, v, option, M, N, "f32", eps=eps)
        return float((r.double() * cr.double()).sum() + (h.double() * ch.double()).sum())

    r, h, st = _forward(cuda_lib, a, option, M, N, "f32", eps=eps)
    names = ("y", "gate", "residual", "w_post", "b_post", "scale", "w_pre", "b_pre")
    out = {k: torch.empty_like(a[k]) for k in names}
    cuda_lib.dlrm_block_norm_bwd(cr, ch, a["y"], a["gate"], r, st, a["w_post"], a["b_post"], a["scale"], a["w_pre"],
                                 *out.values(), workspace=_ws(cuda_lib.dlrm_block_norm_bwd_workspace_size(r)),
                                 **_codes(cuda_lib, option))
    for k in names:
        v, h = _rand(g, *a[k].shape, std=0.5), 2.0**-6
        quotient = (loss(dict(a, **{k: a[k] + h * v})) - loss(dict(a, **{k: a[k] - h * v}))) / (2 * h)
        terms = (out[k].double() * v.double())
        assert abs(quotient - float(terms.sum())) <= 0.005 * float(terms.abs().sum()) + 1e-3, k


# ------------------------------------------------------------------------------------------- choice and order
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,k,pad", [(1, 1, 1, 0), (3, 2, 2, 0), (48, 64, 6, 0), (5, 7, 3, 3), (130, 256, 8, 0),
                                       (33, 255, 1, 1), (2000, 33, 4, 0), (300, 8, 8, 0), (40, 128, 8, 0)])
@pytest.mark.parametrize("closed", [0.0, 0.4, 0.97])
def test_route(cuda_lib, dtype, T, E, k, pad, closed):
    g = torch.Generator().manual_seed(T + E)
    logits = _rand(g, T, E, std=2.0, dtype=dtype, pad=pad)
    if E > 8:
        logits[:, 3] = logits[:, 5]                    # equal ones
    logits[torch.rand(T, E, generator=g).to(dev()) < closed] = -INF
    ids, probs = torch.full((T, k), 9, dtype=torch.int32, device=dev()), torch.empty(T, k, device=dev())
    cuda_lib.dlrm_route_fwd(logits, ids, probs)
    rid, rp = ref.route(_d(logits), k)
    assert torch.equal(ids.cpu().long(), rid)
    assert ((_d(probs) - rp).abs() <= 2.0**-20 * rp).all()
    gp = _rand(g, T, k, std=0.1)
    grad = _empty(T, E, dtype, pad)
    cuda_lib.dlrm_route_bwd(gp, ids, probs, grad)
    p, d = _d(probs), _d(gp)
    dot = (p * d).sum(1, keepdim=True)
    v = p * (d - dot)
    e = p * ((k + 2) * ref.OP * ((p * d).abs().sum(1, keepdim=True) + d.abs()))
    put = lambda t: torch.zeros(T, E + 1, dtype=torch.float64).scatter_(1, torch.where(rid < 0, E, rid), t)[:, :E]
    dref.assert_close(grad, put(v), put(e), dtype)
    assert _guard_ok(grad)


def test_route_gradient_of_the_same_expert_twice(cuda_lib):
    """Not what the choice gives, but what a call may hold: the last of equal ids counts, ids outside none."""
    ids = torch.tensor([[3, 3, 1], [7, -1, 7], [0, 8, 9]], dtype=torch.int32, device=dev())
    probs, gp = torch.rand(3, 3, device=dev()), torch.rand(3, 3, device=dev())
    inside = (ids >= 0) & (ids < 8)
    p, g = torch.where(inside, probs, 0.0).double().cpu(), torch.where(inside, gp, 0.0).double().cpu()
    d = p * (g - (p * g).sum(1, keepdim=True))
    for pad in (0, 1):
        grad = _empty(3, 8, "f32", pad)
        cuda_lib.dlrm_route_bwd(gp, ids, probs, grad)
        want = torch.zeros(3, 8, dtype=torch.float64)
        want[0, 3], want[0, 1], want[1, 7], want[2, 0] = d[0, 1], d[0, 2], d[1, 2], d[2, 0]
        assert ((grad.double().cpu() - want).abs() <= 2.0**-20).all() and _guard_ok(grad)


def test_route_where_logits_are_not_numbers(cuda_lib):
    logits = torch.zeros(6, 40, device=dev())
    logits[0, 11] = NAN
    logits[1, ::3] = -0.0
    logits[2, 4], logits[2, 9] = INF, -INF
    logits[3] = -INF
    logits[4] = -INF
    logits[4, 30] = torch.finfo(torch.float32).min  # the lowest number is open
    logits[5] = torch.finfo(torch.float32).min
    ids, probs = torch.empty(6, 8, dtype=torch.int32, device=dev()), torch.empty(6, 8, device=dev())
    cuda_lib.dlrm_route_fwd(logits, ids, probs)
    assert ids.tolist() == [[11] + list(range(7)), list(range(8)), [4, 0, 1, 2, 3, 5, 6, 7], [-1] * 8, [30] + [-1] * 7,
                            list(range(8))]
    assert probs[0].isnan().all() and (probs[1] == 0.125).all() and probs[2].isnan().all() and (probs[3] == 0).all()
    assert probs[4].tolist() == [1.0] + [0.0] * 7 and (probs[5] == 0.125).all()
    grad = torch.full((6, 40), 7.0, device=dev())
    cuda_lib.dlrm_route_bwd(torch.ones(6, 8, device=dev()), ids, probs, grad)
    assert (grad[3] == 0).all() and (grad[4] == 0).all() and grad[1].abs().max() <= 2.0**-22


@pytest.mark.parametrize("T,k,E,out", [(0, 2, 5, 0.0), (1, 1, 1, 0.0), (31, 1, 3, 0.1), (48, 6, 64, 0.0), (513, 8, 256, 0.2),
                                       (4096, 1, 7, 0.1), (4097, 1, 16, 0.0), (33333, 3, 256, 0.1), (65536, 4, 64, 0.0),
                                       (150001, 8, 33, 0.05), (9000, 2, 4, 1.0)])
def test_sort(cuda_lib, T, k, E, out):
    g = torch.Generator().manual_seed(T + E)
    ids = (torch.randn(T, k, generator=g).abs() * E / 3).long().clamp(max=E - 1)     # unevenly
    none = torch.rand(T, k, generator=g) < out
    ids[none] = -1 - torch.randint(0, 3, (int(none.sum()),), generator=g)
    ids = ids.to(torch.int32).to(dev())
    n = T * k
    off, slots, order = (torch.full(s, 77, dtype=torch.int32, device=dev()) for s in ((E + 1,), (T, k), (n,)))
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    ws = _ws(cuda_lib.dlrm_expert_sort_workspace_size(ids, E))
    cuda_lib.dlrm_expert_sort(ids, E, off, slots, order, workspace=ws, status=status)
    flat = ids.cpu().long().reshape(-1)
    key = torch.where(flat >= 0, flat, E)
    want = torch.argsort(key, stable=True)
    valid = int((flat >= 0).sum())
    place = torch.empty(n, dtype=torch.int64)
    place[want] = torch.arange(n)
    assert torch.equal(slots.cpu().long().reshape(-1), torch.where(flat >= 0, place, -1))
    want[valid:] = -1
    assert torch.equal(order.cpu().long(), want)
    assert off.tolist() == [int((flat[flat >= 0] < e).sum()) for e in range(E + 1)]
    assert status.item() == 0
    if n < 2000 and n:
        assert (off.tolist(), slots.tolist(), order.tolist()) == ref.sort(ids.tolist(), E)
    again = torch.empty_like(slots)
    cuda_lib.dlrm_expert_sort(ids, E, off, again, workspace=ws)
    assert torch.equal(again, slots)


def test_sort_tells_of_experts_that_are_not_there(cuda_lib):
    ids = torch.tensor([[0, 5], [4, -1], [2**31 - 1, 1]], dtype=torch.int32, device=dev())
    off, slots, order = (torch.empty(s, dtype=torch.int32, device=dev()) for s in ((6,), (3, 2), (6,)))
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    cuda_lib.dlrm_expert_sort(ids, 5, off, slots, order, status=status)
    assert status.item() == cuda_lib.DLRM_STATUS_OOB_INDEX
    assert slots.tolist() == [[0, -1], [2, -1], [-1, 1]] and order.tolist() == [0, 5, 2, -1, -1, -1]
    assert off.tolist() == [0, 1, 2, 2, 2, 3]


# ------------------------------------------------------------------------------------------- rows
ROWS = [(1, 1, 1, 0, 0), (1, 8, 4096, 0, 0), (3, 2, 7, 3, 1), (5, 3, 515, 0, 0), (64, 4, 480, 8, 0), (700, 2, 1024, 0, 0),
        (2, 5, 2052, 0, 1), (1300, 8, 40, 0, 0), (900, 1, 33, 0, 0), (40, 8, 3000, 0, 0)]


def _rows_case(seed, T, k, H, pad, lead, dtype, lost):
    g = torch.Generator().manual_seed(seed)
    E = 5
    ids = torch.randint(0, E, (T, k), generator=g)
    ids[torch.rand(T, k, generator=g) < lost] = -1
    _, slots, _ = ref.sort(ids.tolist(), E)
    kw = dict(dtype=dtype, pad=pad, lead=lead)
    return g, kw, torch.tensor(slots, dtype=torch.int32).view(T, k).to(dev())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,H,pad,lead", ROWS)
@pytest.mark.parametrize("lost", [0.0, 0.3])
def test_rows_to_their_experts_and_back(cuda_lib, dtype, T, k, H, pad, lead, lost):
    g, kw, slots = _rows_case(T + H, T, k, H, pad, lead, dtype, lost)
    R = T * k + 2
    at = slots.cpu().long().reshape(-1)
    here = torch.nonzero(at >= 0)[:, 0]
    named = torch.zeros(R, dtype=torch.bool)
    named[at[here]] = True
    token = here // k
    x, res, ys = _rand(g, T, H, **kw), _rand(g, T, H, **kw), _rand(g, R, H, **kw)
    ys[~named.to(dev())] = NAN                          # rows of nobody are not read
    probs = torch.rand(T, k, generator=g).to(dev())
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    # there
    xs = _empty(R, H, dtype, pad, lead)
    cuda_lib.dlrm_dispatch_fwd(x, slots, xs, status=status)
    want = torch.full((R, H), 7.0, dtype=torch.float64)
    want[at[here]] = _d(x)[token]
    assert torch.equal(_d(xs), want) and _guard_ok(xs)
    # the sum back
    gx = _empty(T, H, dtype, pad, lead)
    cuda_lib.dlrm_dispatch_bwd(ys, slots, gx, status=status)
    add = lambda v: torch.zeros(T, v.shape[1], dtype=torch.float64).index_add_(0, token, v)
    rows = _d(ys)[at[here]]
    dref.assert_close(gx, add(rows), (k + 1) * ref.SUM * add(rows.abs()), dtype, "grad_x")
    # weighted, with and without the residual
    p = _d(probs).reshape(-1)[here][:, None]
    for r in (None, res):
        y = _empty(T, H, dtype, pad, lead)
        cuda_lib.dlrm_combine_fwd(ys, slots, probs, r, y, status=status)
        v, size = add(rows * p), add((rows * p).abs())
        if r is not None:
            v, size = v + _d(r), size + _d(r).abs()
        dref.assert_close(y, v, (k + 2) * ref.SUM * size, dtype, "y")
        assert _guard_ok(y)
    # its gradient
    gy, gys, gp = _rand(g, T, H, std=0.1, **kw), _empty(R, H, dtype, pad, lead), torch.full((T, k), 7.0, device=dev())
    cuda_lib.dlrm_combine_bwd(gy, ys, slots, probs, gys, gp, status=status)
    want, bound = torch.full((R, H), 7.0, dtype=torch.float64), torch.zeros(R, H, dtype=torch.float64)
    want[at[here]] = _d(gy)[token] * p
    bound[at[here]] = ref.OP * want[at[here]].abs()
    dref.assert_close(gys, want, bound, dtype, "grad_ys")
    assert _guard_ok(gys)
    v, size = torch.zeros(T * k, dtype=torch.float64), torch.zeros(T * k, dtype=torch.float64)
    v[here], size[here] = (rows * _d(gy)[token]).sum(1), (rows * _d(gy)[token]).abs().sum(1)
    dref.assert_close(gp.view(-1), v, (H + 8) * ref.SUM * size, "f32", "grad_probs")
    one, two = _empty(R, H, dtype, pad, lead), torch.empty_like(gp)
    cuda_lib.dlrm_combine_bwd(gy, None, slots, probs, one, None)
    cuda_lib.dlrm_combine_bwd(gy, ys, slots, None, None, two)
    assert torch.equal(one, gys) and torch.equal(two, gp) and status.item() == 0


def test_rows_that_are_not_there(cuda_lib):
    """Places past the rows are passed over and told of."""
    slots = torch.tensor([[0, 3], [7, -1], [2**31 - 1, 1], [2, -2**31]], dtype=torch.int32, device=dev())
    x, probs = torch.randn(4, 24, device=dev()), torch.rand(4, 2, device=dev())
    for R in (3, 0):
        rows = torch.randn(R, 24, device=dev())
        xs, y, gx, gys, gp = torch.full((R, 24), 7.0, device=dev()), torch.empty(4, 24, device=dev()), torch.empty(4, 24, device=dev()), \
            torch.full((R, 24), 7.0, device=dev()), torch.empty(4, 2, device=dev())
        for call in (lambda s: cuda_lib.dlrm_dispatch_fwd(x, slots, xs, status=s),
                     lambda s: cuda_lib.dlrm_dispatch_bwd(rows, slots, gx, status=s),
                     lambda s: cuda_lib.dlrm_combine_fwd(rows, slots, probs, None, y, status=s),
                     lambda s: cuda_lib.dlrm_combine_bwd(x, rows, slots, probs, gys, gp, status=s)):
            status = torch.zeros(1, dtype=torch.int32, device=dev())
            call(status)
            assert status.item() == cuda_lib.DLRM_STATUS_OOB_INDEX
        if R == 0:
            assert (y == 0).all() and (gx == 0).all() and (gp == 0).all()
            continue
        assert torch.equal(xs, x[[0, 2, 3]]) and torch.equal(gx, torch.stack((rows[0], 0 * rows[0], rows[1], rows[2])))
        assert torch.equal(y[1], 0 * y[1]) and gp[[0, 1, 1, 2, 3], [1, 0, 1, 0, 1]].tolist() == [0.0] * 5
        assert torch.equal(gys, x[[0, 2, 3]] * probs[[0, 2, 3], [0, 1, 0]][:, None])


# ------------------------------------------------------------------------------------------- 8 bits
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,pad,lead", [(1, 1, 0, 0), (3, 7, 3, 1), (5, 32, 0, 0), (2, 33, 0, 0), (9, 100, 8, 0), (700, 480, 0, 0),
                                          (64, 1024, 8, 8), (2, 4099, 0, 0)])
def test_8_bits_there_and_back(cuda_lib, dtype, M, N, pad, lead):
    g = torch.Generator().manual_seed(M + N)
    x = _rand(g, M, N, dtype=dtype, pad=pad, lead=lead)
    wide = torch.exp2(torch.randint(-24 if dtype == "f16" else -140, 16 if dtype == "f16" else 128, (M, -(-N // 32)), generator=g).double())
    spread = torch.exp2(torch.randint(-12, 1, (M, N), generator=g).double())
    top = LARGEST["f16"] if dtype == "f16" else 3.4028234e38
    v = (_d(x) * wide.repeat_interleave(32, 1)[:, :N] * spread).clamp(-top, top)
    x.copy_(v.to(x.dtype).to(dev()))
    if M > 1:
        x[1] = 0.0
    q = torch.full((M, N + pad), 7, dtype=torch.uint8, device=dev())[:, :N]
    e = torch.full((M, -(-N // 32)), 7, dtype=torch.uint8, device=dev())
    cuda_lib.dlrm_pack8(x, q, e)
    rq, re = ref.pack8(_d(x))
    assert torch.equal(e.cpu().long(), re) and torch.equal(q.cpu().long(), rq)
    assert pad == 0 or (q._base[:, N:] == 7).all()
    y = _empty(M, N, dtype, pad, lead)
    cuda_lib.dlrm_unpack8(q, e, y)
    # bf16 rounds the largest numbers of the draw to infinities, which read back as NaN
    got, want, fine = _d(y), ref.unpack8(rq, re, LARGEST[dtype]).to(y.dtype).double(), _d(x).isfinite()
    assert torch.equal(got[fine], want[fine]) and got[~fine].isnan().all() and _guard_ok(y)
    # at most half a step of four bits off, but for the least values and the largest
    size = _d(x).abs()
    off = torch.where(fine, (got - _d(x)).abs(), 0.0)
    assert (off <= torch.maximum(size * 2.0**-4, 2.0**-10 * torch.exp2(re.double() - 127).repeat_interleave(32, 1)[:, :N])).all()


def test_8_bits_of_numbers_that_are_none(cuda_lib):
    for dtype in DTYPES:
        x = torch.zeros(3, 64, dtype=dref.TYPES[dtype], device=dev())
        x[0, 3], x[0, 4], x[0, 5], x[0, 6] = INF, -INF, NAN, 3.0
        x[1, 40] = torch.finfo(x.dtype).max
        x[1, 41] = -torch.finfo(x.dtype).max
        x[2] = float(torch.finfo(x.dtype).smallest_normal) * 2.0**-7
        q, e, y = torch.empty(3, 64, dtype=torch.uint8, device=dev()), torch.empty(3, 2, dtype=torch.uint8, device=dev()), torch.empty_like(x)
        cuda_lib.dlrm_pack8(x, q, e)
        cuda_lib.dlrm_unpack8(q, e, y)
        rq, re = ref.pack8(_d(x))
        assert torch.equal(q.cpu().long(), rq) and torch.equal(e.cpu().long(), re)
        assert y[0, 3:6].isnan().all() and y[0, 6] == 3.0 and (y[0, 7:] == 0).all() and (y[0, :3] == 0).all()
        assert y[1, 40] == LARGEST[dtype] and y[1, 41] == -LARGEST[dtype]
        assert torch.equal(_d(y[2]), ref.unpack8(rq, re, LARGEST[dtype])[2])


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_code_read_back(cuda_lib, dtype):
    q = torch.arange(256, dtype=torch.uint8, device=dev()).repeat(255, 1)
    e = torch.arange(255, dtype=torch.uint8, device=dev())[:, None].repeat(1, 8).contiguous()
    y = torch.empty(255, 256, dtype=dref.TYPES[dtype], device=dev())
    cuda_lib.dlrm_unpack8(q, e, y)
    want = ref.unpack8(q.cpu(), e.cpu(), LARGEST[dtype]).to(y.dtype)
    assert torch.equal(y.isnan().cpu(), want.isnan()) and torch.equal(y.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


BWD8 = [(5, 24, 40), (64, 512, 480), (256, 512, 1024), (1, 40, 13), (1000, 33, 65), (2050, 264, 136), (700, 8, 100), (300, 1, 256),
        (20000, 16, 40)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", BWD8)
@pytest.mark.parametrize("act,p", [("relu", 0.25), ("gelu", 0.0), ("silu", 0.1), ("none", 0.0)])
def test_layer_gradient_from_8_bits(cuda_lib, dtype, M, N, K, act, p):
    """The gradients of the values that the bits stand for: dlrm_linear_bwd's bounds; 2-byte types
    dlrm_linear_bwd's own bits."""
    g = torch.Generator().manual_seed(M + N + K)
    dy, x, z = _rand(g, M, N, std=0.1, dtype=dtype), _rand(g, M, K, dtype=dtype, pad=3), _rand(g, M, N, dtype=dtype)
    w = _rand(g, N, K, std=K**-0.5, dtype=dtype)
    u8 = dict(dtype=torch.uint8, device=dev())
    xq, xe, zq, ze = torch.empty(M, K, **u8), torch.empty(M, -(-K // 32), **u8), torch.empty(M, N, **u8), torch.empty(M, -(-N // 32), **u8)
    cuda_lib.dlrm_pack8(x, xq, xe)
    cuda_lib.dlrm_pack8(z, zq, ze)
    cuda_lib.dlrm_unpack8(xq, xe, x)
    cuda_lib.dlrm_unpack8(zq, ze, z)
    seed, offset = 12345, 2**33 + 1
    rng, code = torch.tensor([seed, offset], device=dev()), dref.ACT[act]
    if act == "none":
        zq = ze = None
    got = [torch.full(s, 7.0, dtype=t, device=dev()) for s, t in (((M, K), dy.dtype), ((N, K), dy.dtype), ((N,), torch.float32))]
    ws = _ws(cuda_lib.dlrm_linear_bwd8_workspace_size(dy, xq, w, act=code, p=p))
    cuda_lib.dlrm_linear_bwd8(dy, xq, xe, w, zq, ze, *got, act=code, p=p, rng=rng, workspace=ws)
    kept, scale = dref.keep_scale(seed, offset, M, N, p) if p else (None, 1.0)
    want = dref.linear_bwd(_d(dy), _d(x), _d(w), _d(z), act, dref.U[dtype], kept, scale)
    for t, k in zip(got, ("dx", "dw", "db")):
        dref.assert_close(t, *want[k], "f32" if k == "db" else dtype, k)
    if dtype != "f32":
        same = [torch.empty_like(t) for t in got]
        cuda_lib.dlrm_linear_bwd(dy, x, w, z, *same, act=code, p=p, rng=rng,
                                 workspace=_ws(cuda_lib.dlrm_linear_bwd_workspace_size(dy, x, w, act=code, p=p)))
        assert all(torch.equal(a, b) for a, b in zip(got, same))
    for i in range(3):                # each alone
        alone = [None] * 3
        alone[i] = torch.empty_like(got[i])
        cuda_lib.dlrm_linear_bwd8(dy, xq if i == 1 else None, xe if i == 1 else None, w, zq, ze, *alone, act=code, p=p, rng=rng,
                                  workspace=ws)
        if i < 2:
            assert torch.equal(alone[i], got[i])
        else:
            dref.assert_close(alone[i], *want["db"], "f32", "db")


def test_layer_gradient_from_8_bits_off_the_grid_and_without_rows(cuda_lib):
    g = torch.Generator().manual_seed(9)
    M, N, K = 77, 51, 91
    dy, w = _rand(g, M, N, std=0.1, dtype="f16", pad=2, lead=1), _rand(g, N, K, dtype="f16", pad=1, lead=3)
    u8 = dict(dtype=torch.uint8, device=dev())
    xq, xe = torch.randint(0, 120, (M, K + 5), **u8)[:, 3:3 + K], torch.randint(118, 124, (M, 3), **u8)
    zq, ze = torch.randint(0, 120, (M, N + 5), **u8)[:, 2:2 + N], torch.randint(118, 124, (M, 2), **u8)
    x, z = torch.empty(M, K, device=dev()).half(), torch.empty(M, N, device=dev()).half()
    cuda_lib.dlrm_unpack8(xq, xe, x)
    cuda_lib.dlrm_unpack8(zq, ze, z)
    out = [torch.empty(M, K, device=dev()).half(), torch.empty(N, K, device=dev()).half(), torch.empty(N, device=dev())]
    same = [torch.empty_like(t) for t in out]
    cuda_lib.dlrm_linear_bwd8(dy, xq, xe, w, zq, ze, *out, act=2,
                              workspace=_ws(cuda_lib.dlrm_linear_bwd8_workspace_size(dy, xq, w, act=2)))
    cuda_lib.dlrm_linear_bwd(dy, x, w, z, *same, act=2, workspace=_ws(cuda_lib.dlrm_linear_bwd_workspace_size(dy, x, w, act=2)))
    assert all(torch.equal(a, b) for a, b in zip(out, same))
    cuda_lib.dlrm_linear_bwd8(dy[:0], xq[:0], xe[:0], w, zq[:0], ze[:0], out[0][:0], out[1], out[2], act=2)
    assert (out[1] == 0).all() and (out[2] == 0).all()
