"""The layer gradient from 8 bits at the bottom of their range (include/dlrm_block.h): blocks with the least
exponent bytes hold values below bf16's least number."""

import pytest
import torch

import block_ref as ref
import dense_ref as dref
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(64, 24, 40), (700, 33, 65), (256, 512, 96), (64, 16, 40), (900, 3, 70), (20000, 1, 33)])
@pytest.mark.parametrize("least", [0, 3])
def test_least_exponents(cuda_lib, M, N, K, least):
    """fp32, gradients of 2^100, so that the sums are ordinary numbers.  Up to 16 outputs the values are taken as they
    are; more outputs multiply them as bf16 numbers, multiples of 2^-133: off by 2^-134 at most, and by
    nothing from an exponent byte of 3 on."""
    g = torch.Generator().manual_seed(M + N + least)
    dy = (torch.randn(M, N, generator=g, dtype=torch.float64) * 2.0**100).float()
    w = torch.randn(N, K, generator=g)
    q = torch.randint(0, 127, (M, K), generator=g) + 128 * torch.randint(0, 2, (M, K), generator=g)
    e = torch.randint(least, least + 4, (M, -(-K // 32)), generator=g)
    x = ref.unpack8(q, e, 3.3895313892515355e38)
    assert float(x[x != 0].abs().min()) < 2.0**-130
    dq, de, ddy, dw = q.to(torch.uint8).to(dev()), e.to(torch.uint8).to(dev()), dy.to(dev()), w.to(dev())
    got = [torch.full(s, 7.0, device=dev()) for s in ((M, K), (N, K), (N,))]
    n = cuda_lib.dlrm_linear_bwd8_workspace_size(ddy, dq, dw)
    cuda_lib.dlrm_linear_bwd8(ddy, dq, de, dw, None, None, *got, workspace=torch.empty(n, dtype=torch.uint8, device=dev()) if n else None)
    want = dref.linear_bwd(dy.double(), x, w.double(), None, "none", dref.U["f32"])
    cut = 2.0**-134 * dy.double().abs().sum(0)[:, None] if N > 16 and least < 3 else 0.0
    for t, k in zip(got, ("dx", "dw", "db")):
        v, bound = want[k]
        dref.assert_close(t, v, bound + (cut if k == "dw" else 0.0), "f32", k)
