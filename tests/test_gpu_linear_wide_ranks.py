"""GPU test of the decode kernels (up to 16 rows) with adapters so wide that rows x rank passes what one round of partial sums holds
(2048 and 4096 floats), against 64 bits: tolerance of the decode kernels, 1e-3 S + 1e-5 and half a bf16 ulp."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import BF, F32, Train, close  # noqa: E402


@pytest.mark.parametrize("M", [2, 7, 9, 13, 16])
@pytest.mark.parametrize("r", [128, 232, 257, 300, 512, 1000, 2048])
@pytest.mark.parametrize("K,bits", [(320, 4), (4096, 3), (16384, 4)])
def test_rows_times_rank(M, r, K, bits):
    print(f"wide decode M={M} r={r} K={K} bits={bits}", flush=True)
    L = Train(M, 72, K, bits, r, seed=M + r, p=0.0)
    L.scale = 16.0 / r
    ref, S = L.linear(0)
    ys = [qlr.linear(L.xd, L.qw, L.Ad, L.Bd, L.scale, out_dtype=o) for o in (BF, F32)]
    ys.append(qlr.linear_dropout(L.xd, L.qw, L.Ad, L.Bd, L.scale))
    torch.cuda.synchronize()
    for y in ys:
        close(y, ref, 1e-3 * S + 1e-5, "y")
    L.p = 0.2
    y = qlr.linear_dropout(L.xd, L.qw, L.Ad, L.Bd, L.scale, L.drop())
    torch.cuda.synchronize()
    ref, S = L.linear(0)
    close(y, ref, 1e-3 * S + 1e-5, "y under a mask")
