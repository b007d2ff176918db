"""GPU test of input gradients whose 256 x 256 tiles fill one round (192 to 256 of them, up to 2048 rows) and run on the tiled
product: against 64 bits, tolerances of the ordinary sizes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import BF, F32, Train, close  # noqa: E402


@pytest.mark.parametrize("M,K", [(1537, 7040), (2048, 8192), (1800, 8000)])
@pytest.mark.parametrize("r,p", [(0, 0.0), (40, 0.0), (40, 0.2)])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_one_round(M, K, r, p, out):
    print(f"round M={M} K={K} r={r} p={p}", flush=True)
    for sides, N in ((1, 8200), (2, 4104)):
        L = Train(M, N, K, 4, r, seed=M + r, sides=sides, p=p)
        if sides == 1:
            got = qlr.linear_dropout_bwd(L.dyd, L.xd, L.qw, L.Ad, L.Bd, L.scale, L.drop(), dx_dtype=out)
            (dx, Sx), a, b = L.grads(0, L.dy.double())
        else:
            got = qlr.gated_bwd(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale, "silu", L.drop(), dx_dtype=out)
            (dx, Sx), a, b = L.gated_grads("silu")
        close(got[0], dx, 5e-3 * sides * Sx + 1e-5, "dx")
        if r:
            close(got[1], a[0], 1e-4 * a[1] + 1e-6, "dA")
            close(got[2], b[0], 1e-4 * b[1] + 1e-6, "dB")
