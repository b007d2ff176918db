"""Host-side test: of up to 16 rows the partial sums of x A^T are no more than the decode kernels behind hold at once (2048 floats a
side of the gated block, 4096 of the layer), read off the workspace sizes; otherwise each output reads them from memory."""
import pytest

from quantized_base_fine_amd import qlr

ROWS, RANKS, COLS = [1, 2, 3, 5, 8, 13, 16], [1, 8, 16, 24, 64, 128], [64, 1024, 4096, 8192, 65536]


def t_bytes(op, M, N, K, r):
    return qlr.workspace_bytes(op, M, N, K, r) - qlr.workspace_bytes(op, M, N, K, 0)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("r", RANKS)
def test_partial_sums_fit_the_decode_kernels(M, r):
    for K in COLS:
        one = lambda sides: sides * M * r * 4  # noqa: E731
        up = lambda b: (b + 255) // 256 * 256  # noqa: E731
        assert up(one(2)) <= t_bytes(qlr.OP_GATED, M, 1024, K, r) <= up(2 * 2048 * 4), K
        assert up(one(1)) <= t_bytes(qlr.OP_LINEAR_DROPOUT, M, 1024, K, r) <= up(4096 * 4), K
