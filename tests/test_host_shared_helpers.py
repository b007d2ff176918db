"""Host-side test: what several kernels share is written once (a change of one copy would miss the other)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_base_fine_amd", "csrc")


def test_shared_pieces_are_defined_once():
    text = "\n".join(open(f).read() for f in sorted(glob.glob(os.path.join(CSRC, "*"))) if os.path.isfile(f))
    for piece in (r"void few_levels\(", r"struct FewTab\b", r"\bkXRow = ", r"[gq]_off\(uint32_t row, uint32_t chunk\) \{\n  const uint32_t h = \(row & 3u\)",
                  r"g?p_off\(uint32_t row, uint32_t chunk\) \{\n  const uint32_t h = \(\(row >> 1\) & 1u\)", r"sharedSizeBytes != 0\) return hipErrorInvalidKernelFile;\n    checked"):
        assert len(re.findall(piece, text)) == 1, piece
