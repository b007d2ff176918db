"""The gated block's decode kernel reads its level table at LDS addresses from 0 and has no static LDS (see
test_host_lds_base).  (No GPU.)"""
import os

from quantized_base_fine_amd import build
from test_host_lds_base import absolute_and_static


def test_the_gated_decode_kernel_has_no_static_lds():
    absolute, bad = absolute_and_static(os.path.join(build.CSRC, "qlr_gated_few.hip"))
    assert len(absolute) == 8 and all("k_gated_few" in k for k in absolute) and not bad
