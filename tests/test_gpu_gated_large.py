"""GPU test of the gated block where a block of 64 elements times its unscaled levels adds up past float32's largest value and g and
v do not: rows whose signs follow a weight row's, and weights of a large scale.  Decode kernel (up to 16 rows) and tiles, against 64
bits; tolerance of the ordinary sizes, 5e-3 S + 1e-5 and half a bf16 ulp."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import BF, F32, close  # noqa: E402

N, K = 72, 128


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("M", [1, 5, 16, 17, 70])
@pytest.mark.parametrize("wscale,xscale", [(0.05, 2.0 ** 125), (4e36, 0.5), (1e-36, 2.0 ** 126), (4e36, 2.0 ** -120), (4e36, 2.0 ** -125)])
def test_sums_before_the_scale(bits, M, wscale, xscale):
    print(f"gated large bits={bits} M={M} w={wscale} x={xscale}", flush=True)
    g = torch.Generator().manual_seed(bits + M)
    qw = qlr.quantize((torch.randn((2 * N, K), generator=g) * wscale).cuda(), bits)
    W = qlr.dequantize(qw, F32).double().cpu()
    n = torch.arange(M) * 5 % (2 * N)                       # row m's signs follow weight row n[m]'s
    x = (torch.sign(W[n]) * (0.5 + 0.5 * torch.rand((M, K), generator=g, dtype=torch.float64)) * xscale).to(BF)
    gu = qlr.gated(x.cuda(), qw, out_dtype=F32, save=True)[1]
    torch.cuda.synchronize()
    ref, S = x.double() @ W.t(), x.double().abs() @ W.abs().t()
    assert (S < 3e38).all()
    close(gu, ref, 5e-3 * S + 1e-5, "gu")
