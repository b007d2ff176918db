"""GPU test of decode calls whose adapter operands fill the rest of a workgroup's 160 KB of LDS to the byte (8-bit codes leave 16 KB): each
runs, against 64 bits with the tolerance of the decode kernels, 1e-3 S + 1e-5 and half a bf16 ulp."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import BF, F32, Train, close  # noqa: E402


# partial sums and t alone; B's rows alone; all three
@pytest.mark.parametrize("M,N,K,r", [(2, 274, 448, 512), (15, 2, 768, 512), (9, 320, 512, 512), (16, 156, 128, 512), (8, 968, 64, 512),
                                     (3, 1048, 896, 128), (8, 104, 64, 496), (8, 104, 64, 504), (8, 104, 64, 520)])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_full_lds(M, N, K, r, out):
    print(f"full LDS M={M} N={N} K={K} r={r}", flush=True)
    L = Train(M, N, K, 8, r, seed=r)
    L.scale = 8.0 / r
    y = qlr.linear(L.xd, L.qw, L.Ad, L.Bd, L.scale, out_dtype=out)
    torch.cuda.synchronize()
    ref, S = L.linear(0)
    close(y, ref, 1e-3 * S + 1e-5, "y")
