"""The dense network's binding refuses tensors that are not on the current device, whichever of the
arguments they are; everything else about them is right.  Nothing here reaches a kernel."""

import ctypes

import pytest
import torch

import dlrm_embeddings_dot_gb300 as dl
from dlrm_embeddings_dot_gb300 import build as libbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()


_never = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: 99)      # stands for the entry points


class Elsewhere:
    """A tensor of the host whose device number is the test's to say."""

    def __init__(self, t, device):
        self.t, self.device_number = t, device

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.device_number


def _calls():
    """(name, function, arguments with every tensor given)"""
    x, w, y = torch.zeros(4, 16), torch.zeros(24, 16), torch.zeros(4, 24)
    b, rng = torch.zeros(24), torch.zeros(2, dtype=torch.int64)
    ws, status = torch.zeros(4096, dtype=torch.uint8), torch.zeros(1, dtype=torch.int32)
    m = torch.zeros(4, 16)
    wr, w1, w2 = torch.zeros(3, 16), torch.zeros(3, 16, 16), torch.zeros(3, 16, 8)
    ids, probs = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    return [
        (dl.dlrm_dropout_fwd, dict(x=x, residual=x, y=m, p=0.1, rng=rng)),
        (dl.dlrm_dropout_bwd, dict(grad_y=x, grad_x=m, p=0.1, rng=rng)),
        (dl.dlrm_linear_fwd, dict(x=x, w=w, bias=b, residual=y, y=y, pre=y, act=1, p=0.1, rng=rng, workspace=ws,
                                  status=status)),
        (dl.dlrm_linear_bwd, dict(grad_y=y, x=x, w=w, pre=y, grad_x=m, grad_w=w, grad_bias=b, act=1, p=0.1, rng=rng,
                                  workspace=ws, status=status)),
        (dl.dlrm_moe_fwd, dict(x=x, w_router=wr, w1=w1, w2=w2, residual=x, y=m, ids=ids, probs=probs, workspace=ws,
                               status=status)),
    ]


CASES = [(i, name) for i, (_, a) in enumerate(_calls()) for name, v in a.items() if isinstance(v, torch.Tensor)]


@pytest.mark.parametrize("i,name", CASES)
def test_host_tensors_are_refused(i, name):
    """All tensors on device 0, so far as they say, but one of the host."""
    call, args = _calls()[i]
    args = {k: Elsewhere(v, 0) if isinstance(v, torch.Tensor) else v for k, v in args.items()}
    args[name] = Elsewhere(args[name].t, -1)
    with pytest.raises(ValueError, match=f"^{name} is not on a CUDA device"):
        _on_device_0(call, args)


@pytest.mark.parametrize("i,name", CASES)
def test_tensors_of_another_device_are_refused(i, name):
    call, args = _calls()[i]
    args = {k: Elsewhere(v, 0) if isinstance(v, torch.Tensor) else v for k, v in args.items()}
    args[name] = Elsewhere(args[name].t, 1)
    with pytest.raises(ValueError, match=f"^{name} is on device 1, not on the current one"):
        _on_device_0(call, args)


def _on_device_0(call, args):
    """The call with a binding whose current device is 0 and whose entry points are never reached."""
    from dlrm_embeddings_dot_gb300 import dense
    m = dense._load()
    at = ctypes.cast(_never, ctypes.c_void_p).value
    m.bind(dense._TYPES, lambda: 0, lambda d: 0, (at,) * 5)
    try:
        call(**args)
    finally:
        dense._marshal = None
        dense._load()


def test_plain_host_tensors_are_refused():
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="not on a CUDA device"):
        dl.dlrm_dropout_fwd(x, None, torch.zeros(4, 16), 0.1, torch.zeros(2, dtype=torch.int64))


def test_short_status_is_refused():
    x, w, y = torch.zeros(4, 16), torch.zeros(8, 16), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="status"):
        dl.dlrm_linear_fwd(x, w, None, None, y, status=torch.zeros(0, dtype=torch.int32))


@pytest.mark.parametrize("act", [2**32, 2**32 + 1, -2**31 - 1])
def test_activations_past_32_bits_are_refused(act):
    """2^32 + 1 is not RELU."""
    x, w, y = (Elsewhere(torch.zeros(4, 16), 0), Elsewhere(torch.zeros(8, 16), 0), Elsewhere(torch.zeros(4, 8), 0))
    with pytest.raises(ValueError, match="^act is"):
        _on_device_0(dl.dlrm_linear_fwd, dict(x=x, w=w, bias=None, residual=None, y=y, act=act))


@pytest.mark.parametrize("ws", [torch.zeros(1, dtype=torch.uint8).expand(1 << 30), torch.zeros(64, dtype=torch.uint8)[::2]])
def test_workspaces_that_are_not_contiguous_are_refused(ws):
    """An expanded byte says it has a gigabyte."""
    x, w, y = (Elsewhere(torch.zeros(4, 16), 0), Elsewhere(torch.zeros(8, 16), 0), Elsewhere(torch.zeros(4, 8), 0))
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        _on_device_0(dl.dlrm_linear_fwd, dict(x=x, w=w, bias=None, residual=None, y=y, workspace=Elsewhere(ws, 0)))
