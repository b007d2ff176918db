"""GPU test of the double-binary adapter at wide ranks and several envelope terms with up to 16 rows and a few more, against 64 bits:
1e-3 S + 1e-5 (5e-3 S of the tiled kernel, from 17 rows on) and half a bf16 ulp, S the sums of the sizes of the base's and of the branch's terms."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import BF, F32, close  # noqa: E402


def signs(rows, cols, g):
    """(+-1 matrix, its bits in 32-bit words, LSB first)"""
    S = torch.randint(2, (rows, cols), generator=g)
    words = (cols + 31) // 32
    P = torch.zeros((rows, words * 32), dtype=torch.int64)
    P[:, :cols] = S
    v = (P.view(rows, words, 32) << torch.arange(32)).sum(2)
    return (2 * S - 1).double(), torch.where(v >= 2 ** 31, v - 2 ** 32, v).int()


@pytest.mark.parametrize("M", [1, 3, 9, 16, 17, 50])
@pytest.mark.parametrize("R,ell", [(65, 1), (100, 1), (130, 1), (33, 4), (200, 2)])
@pytest.mark.parametrize("N,K,bits", [(59, 192, 8), (104, 1024, 4), (72, 4096, 3)])
def test_wide(M, R, ell, N, K, bits):
    print(f"dba M={M} R={R} l={ell} N={N} K={K} bits={bits}", flush=True)
    g = torch.Generator().manual_seed(M + R + N)
    qw = qlr.quantize((torch.randn((N, K), generator=g) * 0.05).cuda(), bits)
    W = qlr.dequantize(qw, F32).double().cpu()
    x = torch.randn((M, K), generator=g).to(BF)
    (B1, p1), (B2, p2) = signs(N, R, g), signs(R, K, g)
    al, be, ga = [(torch.randn(s, generator=g) * k).half() for s, k in (((ell, N), 0.3), ((ell, R), R ** -0.5), ((ell, K), K ** -0.5))]
    ref, S, xd = x.double() @ W.t(), x.double().abs() @ W.abs().t(), x.double()
    for i in range(ell):
        z = (xd * ga[i].double()) @ B2.t()
        ref = ref + ((z * be[i].double()) @ B1.t()) * al[i].double()
        S = S + torch.outer((xd.abs() @ ga[i].double().abs()) * be[i].double().abs().sum(), al[i].double().abs())
    for out in (BF, F32):
        y = qlr.linear_dba(x.cuda(), qw, p1.cuda(), p2.cuda(), al.cuda(), be.cuda(), ga.cuda(), out_dtype=out)
        torch.cuda.synchronize()
        close(y, ref, (1e-3 if M <= 16 else 5e-3) * S + 1e-5, "y")
