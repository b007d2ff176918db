"""Host-side test of what the header says the workspaces of the calls under adapter dropout and of the gated block hold."""
import os
import re

import pytest

from quantized_base_fine_amd import qlr

D, DB, G, GB = qlr.OP_LINEAR_DROPOUT, qlr.OP_LINEAR_DROPOUT_BWD, qlr.OP_GATED, qlr.OP_GATED_BWD
ws = qlr.workspace_bytes


def test_no_rows_or_no_adapter():
    for op in (D, DB, G, GB):
        assert ws(op, 0, 1024, 1024, 16) == 0
    for M in (1, 16, 17, 64, 2048):
        assert ws(D, M, 1024, 1024, 0) == 0


def test_parts_without_an_adapter():
    """Sums of ranges of the contraction (a multiple of one range's, at most 8), and the copy of the weight."""
    for M, N, K in ((1, 4096, 4096), (64, 1024, 1024), (333, 520, 4096)):
        for op, cols in ((G, 2 * N), (DB, K), (GB, K)):
            dgu = M * 2 * N * 2 if op == GB else 0
            sums = ws(op, M, N, K, 0) - (dgu + 255) // 256 * 256
            assert sums % (M * cols * 4) == 0 and sums // (M * cols * 4) <= 8, (op, M, N, K)
            assert sums > 0 or M == 333, (op, M, N, K)  # (its backward's 9 steps are not split)
    assert ws(G, 64, 1024, 1024, 0) == 4 * 64 * 2048 * 4
    assert ws(G, 2048, 11008, 4096, 0) == 2 * 11008 * 4096 * 2


@pytest.mark.parametrize("M,r", [(1, 0), (64, 0), (2048, 0)])
def test_a_block_without_an_adapter_asks_for_its_workspace(M, r):
    """NULL is refused where the size is not 0."""
    w = qlr.C.byref(qlr.CQWeight(1, 4, 64, 256, 2 * 11008, 4096, 1 << 24, 2 << 24, 3 << 24))
    call = qlr.lib().qlr_gated_fwd(4 << 24, qlr.QLR_BF16, M, w, 0, None, None, qlr.QLR_BF16, r, 0.0, None, 5 << 34, qlr.QLR_BF16, None,
                                   None, 0, None)
    assert qlr.STATUS[call] == "QLR_ERR_WORKSPACE" and ws(G, M, 11008, 4096, r) > 0


def test_the_header_names_the_parts():
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "qlr.h")).read()
    text = re.sub(r"\s*\n \*\s*", " ", text)
    part = text[text.index("QLR_OP_LINEAR_DROPOUT and QLR_OP_GATED"):text.index("Contents need no")]
    for words in ("bf16 copy of the weight", "ranges of the contraction", "the masks' bits", "without an adapter",
                  "0 bytes when M, N or K is 0, and for QLR_OP_LINEAR_DROPOUT when r is 0"):
        assert words in part, words
