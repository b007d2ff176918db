"""Host-side tests of when the input gradients of many rows go through a dense copy of the weight, and of when a product's contraction is
split, read off the workspace: without an adapter it holds nothing else."""
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


@pytest.mark.parametrize("M,N", [(333, 1403), (333, 2048), (600, 1024), (130, 4096), (64, 11008)])
def test_many_short_tiles_are_not_split(M, N):
    """128 tiles of 64 x 128 and more: unsplit up to 40 steps of 64."""
    for K, split in ((1024, False), (2048, False), (2560, False), (2624, True), (4096, True)):
        assert (qlr.workspace_bytes(qlr.OP_GATED, M, N, K, 0) > 0) == split, K


def test_few_tiles_are():
    for K, split in ((256, False), (512, True), (2048, True), (4096, True)):
        assert (qlr.workspace_bytes(qlr.OP_GATED, 333, 700, K, 0) > 0) == split, K
