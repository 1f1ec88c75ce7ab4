"""The choice of experts and the order of the choices as one follows the other on a stream: choices of more
than one block, written right before they are sorted, replayed with others in their place."""

import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu


def _choose(logits, k):
    """The choice in 64 bits on the host: the largest first, equal ones by lower index (none here)."""
    return torch.topk(logits.double().cpu(), k, dim=1).indices


def _order(ids, E):
    """(offsets, slots, order) of choices that all have an expert."""
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True)
    slots = torch.empty_like(flat)
    slots[order] = torch.arange(len(flat))
    return torch.searchsorted(flat[order], torch.arange(E + 1)), slots.view(ids.shape), order


@pytest.mark.parametrize("T,k,E", [(2100, 2, 6), (9000, 1, 16), (9000, 1, 1), (20011, 3, 40), (65536, 4, 64), (65537, 2, 256)])
def test_choices_sorted_right_behind_the_choice(cuda_lib, T, k, E):
    """One graph of the choice, its order and the rows' way there and back, replayed over logits that change
    in place: the order is always that of the choices just made.  (2100 x 2 are the fewest in two blocks.)"""
    d = dict(device=dev())
    g = torch.Generator().manual_seed(T + E)
    draws = [torch.randn(T, E, generator=g) for _ in range(3)]
    logits = draws[0].to(dev())
    x = torch.arange(T, **d).float()[:, None].repeat(1, 4)
    ids, slots = torch.empty(T, k, dtype=torch.int32, **d), torch.empty(T, k, dtype=torch.int32, **d)
    order, off = torch.empty(T * k, dtype=torch.int32, **d), torch.empty(E + 1, dtype=torch.int32, **d)
    probs, xs, back = torch.empty(T, k, **d), torch.empty(T * k, 4, **d), torch.empty(T, 4, **d)
    status = torch.zeros(1, dtype=torch.int32, **d)
    n = cuda_lib.dlrm_expert_sort_workspace_size(ids, E)
    assert n > 0                                             # more than one block
    ws = torch.empty(n, dtype=torch.uint8, **d)

    def run():
        cuda_lib.dlrm_route_fwd(logits, ids, probs)
        cuda_lib.dlrm_expert_sort(ids, E, off, slots, order, workspace=ws, status=status)
        cuda_lib.dlrm_dispatch_fwd(x, slots, xs, status=status)
        cuda_lib.dlrm_dispatch_bwd(xs, slots, back, status=status)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    want = [(i, *_order(i, E)) for i in (_choose(v, k) for v in draws)]
    for at in (0, 1, 2, 1, 0):
        logits.copy_(draws[at])
        graph.replay()                                       # twice with nothing in between
        graph.replay()
        i, o, s, c = want[at]
        assert torch.equal(ids.cpu().long(), i)
        assert torch.equal(off.cpu().long(), o) and torch.equal(slots.cpu().long(), s) and torch.equal(order.cpu().long(), c)
        assert torch.equal(xs.cpu()[:, 0].long(), c // k) and torch.equal(back.cpu(), k * x.cpu())
    assert status.item() == 0


@pytest.mark.parametrize("E", [1, 2, 3, 256])
@pytest.mark.parametrize("T", [4097, 6144, 70001, 262145])
def test_few_and_many_experts_over_blocks(cuda_lib, T, E):
    """More parts of the counts than blocks, and as many experts as there can be; some choices without expert."""
    g = torch.Generator().manual_seed(T + E)
    ids = torch.randint(-1, E, (T, 1), generator=g)
    dids = ids.to(torch.int32).to(dev())
    off, slots, order = (torch.full(s, 77, dtype=torch.int32, device=dev()) for s in ((E + 1,), (T, 1), (T,)))
    ws = torch.full((cuda_lib.dlrm_expert_sort_workspace_size(dids, E),), 255, dtype=torch.uint8, device=dev())
    cuda_lib.dlrm_expert_sort(dids, E, off, slots, order, workspace=ws)
    key = torch.where(ids[:, 0] >= 0, ids[:, 0], E)
    want = torch.argsort(key, stable=True)
    place = torch.empty(T, dtype=torch.int64)
    place[want] = torch.arange(T)
    here = int((key < E).sum())
    want[here:] = -1
    assert torch.equal(slots.cpu().long()[:, 0], torch.where(key < E, place, -1)) and torch.equal(order.cpu().long(), want)
    assert torch.equal(off.cpu().long(), torch.searchsorted(key.sort().values, torch.arange(E + 1)))
