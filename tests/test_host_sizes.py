"""Host-side tests of the largest sizes of the 8-bit-integer and expert-grouped calls: refused before any launch (every call
below fails its checks)."""
from test_host_i8_grouped import P, bwd, grouped, i8

import pytest


def test_linear_i8_sizes():
    big = (1 << 14, 64, P["w"], P["s"])
    assert i8(M=1 << 27, w=big) == "ERR_SHAPE"                                      # y of 2^41 elements
    assert i8(M=1 << 26, w=(32, 1 << 15, P["w"], P["s"])) == "ERR_SHAPE"            # x of 2^41 elements
    assert i8(M=1 << 26, w=big, wsb=0) == "ERR_ALIAS"                               # 2^40: past the size checks
    assert i8(M=1, w=((1 << 30) + 1, 64, P["w"], P["s"])) == "ERR_SHAPE"


@pytest.mark.parametrize("call", [grouped, bwd], ids=["forward", "backward"])
def test_grouped_sizes(call):
    assert call(T=1 << 27, rows=2 << 14) == "ERR_SHAPE"       # y (dy) of 2^41 elements
    assert call(T=1 << 27, cols=1 << 14) == "ERR_SHAPE"       # x of 2^41 elements
    assert call(T=1, rows=2 * ((1 << 20) + 8)) == "ERR_SHAPE" and call(T=1, cols=(1 << 20) + 64) == "ERR_SHAPE"
