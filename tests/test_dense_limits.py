"""The dense network's entry points at the largest sizes their arguments can name."""

import pytest
import torch

import dense_ref as ref
import dlrm_embeddings_dot_gb300 as dl
from dlrm_embeddings_dot_gb300 import build as libbuild
from gpu_util import dev

FAKE = 0x10000      # never dereferenced
MOST = 2**31 - 1


def test_mixture_refuses_widths_near_2_31():
    libbuild.build()
    L = dl.load()

    def call(H, I, T=1):
        return L.dlrm_moe_fwd(FAKE, H, FAKE, FAKE, FAKE, None, 0, 1, T, H, I, 1, 1, 3, 0, FAKE, H, FAKE, FAKE, FAKE, 1 << 50,
                              None, None)

    for H, I in ((MOST, 1), (MOST - 6, 1), (1, MOST), (MOST - 2**20 + 1, 8)):
        for T in (0, 1):
            assert call(H, I, T) == dl.DLRM_ERR_UNSUPPORTED, (H, I, T)
            assert "dlrm_moe_fwd" in dl.dlrm_last_error()


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
