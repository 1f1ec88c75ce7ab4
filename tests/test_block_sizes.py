"""Workspace sizes by the binding, where not every tensor of a call is there (no GPU is asked)."""

import pytest
import torch

import dlrm_embeddings_dot_gb300 as dl
from dlrm_embeddings_dot_gb300 import build as libbuild


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(64, 24, 40), (5000, 8, 40), (1, 512, 480), (0, 24, 40)])
def test_layer_gradient_without_its_input(dtype, M, N, K):
    """dlrm_linear_bwd8 takes None for the input where grad_w is not asked for, and so does its size."""
    libbuild.build()
    dy, w, x = torch.empty(M, N, dtype=dtype), torch.empty(N, K, dtype=dtype), torch.empty(M, K, dtype=torch.uint8)
    size = dl.dlrm_linear_bwd8_workspace_size(dy, x, w, act=2)
    assert dl.dlrm_linear_bwd8_workspace_size(dy, None, w, act=2) == size and (size > 0 or M == 0)
