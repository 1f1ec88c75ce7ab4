"""Which form a dense layer takes, seen from the workspace it asks for (none where weights or rows are
streamed, fp32 operands laid out again where they run in tiles)."""

import dlrm_embeddings_dot_gb300 as dl
from dlrm_embeddings_dot_gb300 import build as libbuild

FAKE = 0x10000      # never dereferenced


def _tiles(dtype, M, N, K):
    libbuild.build()
    # rows off the 16-byte grid, so that the tiles need copies in every type
    return dl.load().dlrm_linear_fwd_workspace_size(FAKE + 4, K, FAKE + 4, K, dtype, M, N, K) > 0


def test_weights_of_16_mb_are_streamed_for_32_rows_only():
    for dtype, es in ((dl.DLRM_F32, 4), (dl.DLRM_F16, 2), (dl.DLRM_BF16, 2)):
        K = 1024
        at = (1 << 24) // (K * es)                     # outputs whose weights are 16 MB
        for M in (1, 9, 32):
            assert not _tiles(dtype, M, at, K) and not _tiles(dtype, M, 8 * at, K)
        for M in (33, 48, 64):
            assert _tiles(dtype, M, at, K) and not _tiles(dtype, M, at - 1, K)
        assert _tiles(dtype, 65, 64, 64)
