"""Host-side test of when the input gradients of many rows go through a dense copy of the weight, read off the workspace (the copy is
its largest part, and there is nothing else without an adapter)."""
import pytest

from quantized_base_fine_amd import qlr

DB, GB = qlr.OP_LINEAR_DROPOUT_BWD, qlr.OP_GATED_BWD


def copies(op, M, N, K):
    dgu = M * 2 * N * 2 if op == GB else 0
    weight = (2 if op == GB else 1) * N * K * 2
    rest = qlr.workspace_bytes(op, M, N, K, 0) - dgu
    assert rest < 256 or rest >= weight or rest < 8 * M * K * 4 + 256
    return rest >= weight


@pytest.mark.parametrize("op,N", [(DB, 8192), (DB, 11008), (GB, 4096)], ids=["layer", "layer, long", "block"])
def test_one_round_of_tiles_needs_no_copy(op, N):
    """192 to 256 tiles of 256 x 256, up to 2048 rows."""
    for M, K in ((1536, 8192), (1792, 7040), (2048, 6144), (2048, 8192)):
        assert not copies(op, M, N, K), (M, K)


@pytest.mark.parametrize("op,N", [(DB, 8192), (DB, 11008), (GB, 5632)], ids=["layer", "layer, long", "block"])
def test_other_gradients_of_many_rows_do(op, N):
    """Fewer tiles, a second round, or more rows."""
    for M, K in ((1536, 4096), (2048, 4096), (2048, 5632), (2048, 8448), (1536, 11008), (2560, 5632), (4096, 4096), (4096, 8192)):
        assert copies(op, M, N, K), (M, K)
    for M, K in ((1535, 4096), (1024, 8192)):
        assert not copies(op, M, N, K), (M, K)
