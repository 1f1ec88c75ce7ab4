"""Slopes of the residual blocks' gates far from 0 (include/dlrm_block.h): saturated gates keep the digits
of their gradients."""

import pytest
import torch

import block_ref as ref
import dense_ref as dref
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gate", ["sigmoid", "silu"])
@pytest.mark.parametrize("N", [16, 99, 200, 256, 771, 1024])
@pytest.mark.parametrize("per_row", [False, True])
def test_slopes_of_saturated_gates(cuda_lib, dtype, gate, N, per_row):
    """y, its gradient and the kept 1 / sqrt are 1 and the mean 0, so the gate's gradient is its slope (by row: N of them).
    Bound: the exponential's argument is off by 2^-24 of its size for each of its factor and its rounding, so e^-g
    by |g| 2^-23; the hardware's exponential and reciprocal by 2^-22 and 2^-23, the products by
    2^-24 each: |g| 2^-22 + 2^-20 of the slope's factors in all.  |g| up to 80: e^-g is a normal number."""
    t = dref.TYPES[dtype]
    M = 40
    g = torch.linspace(-80, 80, M * (1 if per_row else N), dtype=torch.float64).view(M, -1).to(t).to(dev())
    ones = torch.ones(M, N, dtype=t, device=dev())
    st = torch.tensor([[0.0, 1.0, 0.0, 0.0]], device=dev()).repeat(M, 1)
    out = torch.full_like(g, 7.0)
    cuda_lib.dlrm_block_norm_bwd(ones, None, ones, g, None, st, None, None, None, None, None, out, None, *[None] * 5,
                                 gate_act=ref.GATES[gate])
    v = g.double().cpu()
    s, rest = torch.sigmoid(v), torch.sigmoid(-v)
    slope = s * rest if gate == "sigmoid" else s * (1 + v * rest)
    terms = s * rest if gate == "sigmoid" else s * (1 + v.abs() * rest)
    n = N if per_row else 1
    dref.assert_close(out, n * slope, n * (v.abs() * 2.0**-22 + 2.0**-20) * terms, dtype)
