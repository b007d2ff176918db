"""GPU test of the decode kernels (up to 16 rows) where an adapter's B has an odd number of elements: its last one lies in half a word.
Every column against 64 bits, tolerance of the decode kernels, 1e-3 S + 1e-5 and half a bf16 ulp; the last column is also checked with
an adapter of that element alone."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import BF, F32, Train, close  # noqa: E402


def calls(L):
    yield "linear", lambda: qlr.linear(L.xd, L.qw, L.Ad, L.Bd, L.scale, out_dtype=F32)
    yield "bf16", lambda: qlr.linear(L.xd, L.qw, L.Ad, L.Bd, L.scale, out_dtype=BF)
    yield "static", lambda: qlr.linear_static(L.xd, L.qw, L.Ad, L.Bd, L.scale, out_dtype=F32)
    yield "dropout", lambda: qlr.linear_dropout(L.xd, L.qw, L.Ad, L.Bd, L.scale, out_dtype=F32)
    yield "mixed", lambda: qlr.linear_mixed([dict(x=L.xd, qw=L.qw, A=L.Ad, B=L.Bd, scale=L.scale) for _ in range(2)], out_dtype=F32)[1]


@pytest.mark.parametrize("M", [1, 2, 8, 16])
@pytest.mark.parametrize("N", [1, 17, 59, 333, 4097])
@pytest.mark.parametrize("r", [1, 3, 13, 15, 33])
@pytest.mark.parametrize("K,bits", [(192, 8), (128, 3), (1024, 4), (4096, 4), (1024, 2)])
def test_last_element_of_b(M, N, r, K, bits):
    print(f"odd adapter M={M} N={N} r={r} K={K} bits={bits}", flush=True)
    L = Train(M, N, K, bits, r, seed=M + N + r)
    ref, S = L.linear(0)
    for name, call in calls(L):
        close(call(), ref, 1e-3 * S + 1e-5, name)
    L.B = torch.zeros_like(L.B)
    L.B[-1, -1] = 1.0
    L.Bd = L.B.cuda()
    ref, S = L.linear(0)
    for name, call in calls(L):
        close(call(), ref, 1e-3 * S + 1e-5, name + ", last element alone")


@pytest.mark.parametrize("M", [1, 5])
@pytest.mark.parametrize("N,r", [(59, 3), (333, 15), (17, 1)])
def test_outliers(M, N, r):
    """The same with the side channel of outliers in the kernel (one row) and before it."""
    L = Train(M, N, 1024, 4, r, seed=N)
    W = torch.randn((N, 1024), generator=torch.Generator().manual_seed(3)) * 0.05
    qo, sp = qlr.quantize_outliers(W.cuda(), 4, 30)
    base = qlr.linear_outliers(L.xd, qo, sp, out_dtype=F32).double().cpu()
    y = qlr.linear_outliers(L.xd, qo, sp, L.Ad, L.Bd, L.scale, out_dtype=F32)
    torch.cuda.synchronize()
    x, A, B = L.x.double(), L.A.double(), L.B.double()
    S = L.scale * (x.abs() @ A.abs().t()) @ B.abs().t()
    close(y.double() - base.cuda(), L.scale * (x @ A.t()) @ B.t(), 1e-3 * S + 2e-6 * base.abs() + 1e-5, "the adapter's part")
