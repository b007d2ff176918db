"""GPU tests of tile shapes and borders that the other tests of the 8-bit-integer and expert-grouped calls do not reach:
128 x 128 tiles as a whole call, malformed offsets over long ranges, and the largest integer sums with -128.  Oracles and
tolerances of test_gpu_grouped.py and test_gpu_i8.py."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from test_gpu_grouped import BF, F32, Layer, check_backward, check_forward  # noqa: E402
from test_gpu_i8 import check  # noqa: E402


@pytest.mark.parametrize("m,K,wv,xv", [(3, 131056, -128, -128), (18, 131056, -128, -128), (3, 131072, -128, 127),
                                       (18, 131072, -128, 127), (18, 131072, 127, -128)])
def test_largest_sums_with_minus_128(m, K, wv, xv):
    """128 * 128 * 131056 = 2 147 221 504 < 2^31, the largest K (a multiple of 16) for -128 in both operands."""
    print(f"linear_i8 M={m} K={K} w={wv} x={xv}", flush=True)
    w8, xq = qlr.I8Rows.empty(24, K, "cuda"), qlr.I8Rows.empty(m, K, "cuda")
    w8.q.fill_(wv), xq.q.fill_(xv), w8.scale.fill_(0.5), xq.scale.fill_(0.25)
    y = qlr.linear_i8(None, w8, xq=xq, out_dtype=F32)
    torch.cuda.synchronize()
    ref = torch.full((m, 24), float(wv * xv * K) * 0.125, dtype=torch.float64)
    check(y, ref, 4e-7 * ref.abs())
