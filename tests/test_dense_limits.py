"""The dense network's entry points at the largest sizes their arguments can name."""

import pytest
import torch

import dense_ref as ref
from gpu_util import dev

MOST = 2**31 - 1


@pytest.mark.gpu
@pytest.mark.parametrize("N", [MOST, MOST - 7])
def test_dropout_of_the_widest_row(cuda_lib, N):
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    x = torch.ones(1, N, dtype=torch.float16, device=dev())
    y = torch.empty_like(x)
    rng = torch.tensor([9, 1], dtype=torch.int64, device=dev())
    cuda_lib.dlrm_dropout_fwd(x, None, y, 0.25, rng)
    for col in (0, 5, 2**30 + 3, N - 9, N - 2, N - 1):
        w = ref.philox([col // 8, 0, 1, 0], [9, 0])[(col % 8) // 2]
        kept = (w >> 16 * (col % 2) & 0xFFFF) >= ref.threshold(0.25)
        assert (y[0, col].item() != 0) == kept, col
    share = (y != 0).sum().item() / N
    assert abs(share - 0.75) < 1e-4
