"""GPU test: which kernel a gated block of up to 16 rows runs on by its adapters' rank, by its results' bits: the decode kernel where it
holds the adapters on chip (8, 16 .. 64 columns, or at most 2), the tiles elsewhere."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import F32, Train, close  # noqa: E402


@pytest.mark.parametrize("M", [1, 7, 16])
@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("r", [0, 1, 2, 3, 8, 12, 16, 63, 64, 65, 72, 128])
def test_kernel_by_rank(M, p, r):
    print(f"gated rule M={M} p={p} r={r}", flush=True)
    L = Train(M, 264, 1024, 4, r, seed=M + r, sides=2, p=p if r else 0.0)
    want = qlr.PATH_GEMV if r <= 2 or (r <= 64 and r % 8 == 0) else qlr.PATH_GEMM
    run = lambda: qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale, "silu", L.drop(), out_dtype=F32, save=True)  # noqa: E731
    h, gu = run()
    both = {}
    for path in (qlr.PATH_GEMV, qlr.PATH_GEMM):
        with qlr.path(path):
            both[path] = run()
    torch.cuda.synchronize()
    assert torch.equal(h, both[want][0]) and torch.equal(gu, both[want][1])
    assert not torch.equal(both[qlr.PATH_GEMV][0], both[qlr.PATH_GEMM][0])
    ref, tol, rgu, S = L.gated("silu")
    for hh, gg in both.values():
        close(gg, rgu, 5e-3 * S + 1e-5, "gu")
        close(hh, ref, tol, "h")
