"""Host-side tests of qlr_workspace_bytes for the calls under adapter dropout and the gated block at the sizes that no call
takes: empty weights, and sizes past the calls' limits.  Each op runs in a process of its own, so that one that ends it is a
failure of its test."""
import subprocess
import sys

import pytest

OPS = ["LINEAR_DROPOUT", "LINEAR_DROPOUT_BWD", "GATED", "GATED_BWD"]


def sizes(op, cases):
    """What qlr.workspace_bytes gives for each case: a number, or the name of the error."""
    code = ("from quantized_base_fine_amd import qlr\n"
            f"for c in {cases!r}:\n"
            "    try:\n"
            f"        print(qlr.workspace_bytes(qlr.OP_{op}, *c))\n"
            "    except qlr.QlrError as e:\n"
            "        print(str(e).split()[0].rstrip(':'))\n")
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, (op, p.returncode, p.stderr[-400:])
    return p.stdout.split()


@pytest.mark.parametrize("op", OPS)
def test_empty_weights_need_nothing(op):
    cases = [(M, N, K, r) for M in (0, 1, 16, 17, 2048) for N, K in ((0, 64), (64, 0), (0, 0)) for r in (0, 8, 100)]
    assert sizes(op, cases) == ["0"] * len(cases)


@pytest.mark.parametrize("op", OPS)
def test_sizes_past_the_limits_are_refused(op):
    """M 2^27, N and K 2^20 (the gated block's N 2^19), r 2^20, M N and M K 2^40 (2^39)."""
    gated = op.startswith("GATED")
    n, k, e = (1 << 19) if gated else 1 << 20, 1 << 20, (1 << 39) if gated else 1 << 40
    good = [((1 << 27), 8, 64, 8), (17, n, 64, 8), (17, 8, k, 8), (17, 8, 64, 1 << 20), (e // n, n, 64, 1), (e // k, 8, k, 1)]
    bad = [((1 << 27) + 1, 8, 64, 8), (17, n + 8, 64, 8), (17, 8, k + 64, 8), (17, 8, 64, (1 << 20) + 1), (e // n + 1, n, 64, 1),
           (e // k + 1, 8, k, 1), (1 << 62, 64, 64, 8), (1 << 31, 1 << 31, 1 << 31, 1 << 30), (1 << 62, 1 << 62, 1 << 62, 8),
           ((1 << 63) - 1, (1 << 63) - 1, (1 << 63) - 1, (1 << 31) - 1)]
    got = sizes(op, good + bad)
    assert all(int(g) > 0 for g in got[:len(good)])
    assert all("ERR_SHAPE" in g for g in got[len(good):]), got


def test_plain_backward_of_an_empty_weight():
    """The plain layer's backward: its size without rows and columns is t, u and B transposed alone, as with either of them."""
    got = sizes("LINEAR_BWD", [(M, 0, 0, r) for M in (0, 1, 17, 300) for r in (0, 8, 100)])
    assert [int(g) for g in got] == [0, 0, 0, 0, 512, 1024, 0, 1536, 2 * 6912, 0, 2 * 9728, 2 * 120064]
