"""GPU test of what the levels' rounding costs the gated block's decode: the error of the up projection alone, in relative 2-norm
against 64 bits.  The gate is 30 in every row (a block of ones times one element of x; SiLU of 30 is 30 to 1e-13) and the up
projection has blocks of its own, so that a float32 h is 30 v.

The table holds bf16(f level) with an f for the code width.  With e = bf16(f level) / f - level times the block's scale, output n of a
row x is off by sum_k x_k e_nk, whose square is sum_k e_nk^2 in the mean over independent x_k of variance 1, as v's own is sum_k w_nk^2: the
error in 2-norm over all outputs is |e| / |w| of v's, Frobenius norms over the weight, which the test forms from its codes.  The two norms over
N outputs of a row scatter by 1 / sqrt(2 N) each, 2.2 % at N = 1000: 15 % above it is six times both together.  Float32 sums and scales
add at most 5e-7.  At f = 1 the same quotient is 1.2 to 200 times as large."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import BF, F32  # noqa: E402

UNIT = {2: 1.6640625, 3: 1.1953125, 4: 1.6015625, 8: 1.59375}


def quotient(D, bits, f):
    """|e| / |w| of a weight W' (rows x 64 n): its levels from its blocks' largest elements, whose level is 1 or -1."""
    levels = torch.tensor(qlr.codebook(bits), dtype=torch.float64)
    blocks = D.double().cpu().view(-1, 64)
    scale = blocks.abs().amax(1, keepdim=True)
    w = blocks / scale
    mid = (levels[1:] + levels[:-1]) / 2
    lev = levels[torch.bucketize(w, mid)]
    assert (lev - w).abs().max() < 1e-6
    e = ((f * lev).float().to(BF).double() / f - lev) * scale
    return (e.norm() / blocks.norm()).item()


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("M", [1, 5, 16])
@pytest.mark.parametrize("N", [1000, 9000])
def test_error_of_the_levels(bits, M, N):
    print(f"levels bits={bits} M={M} N={N}", flush=True)
    g = torch.Generator().manual_seed(bits + M)
    W = torch.zeros((2 * N, 64 + 1024))
    W[:N, :64] = 1.0
    W[N:, 64:] = torch.randn((N, 1024), generator=g) * 0.05
    qw = qlr.quantize(W.cuda(), bits)
    D = qlr.dequantize(qw, F32)
    assert (D[:N, :64] == 1).all() and not D[:N, 64:].any() and not D[N:, :64].any()
    x = torch.zeros((M, 64 + 1024))
    x[:, 0], x[:, 64:] = 30.0, torch.randn((M, 1024), generator=g)
    x = x.to(BF)
    h = qlr.gated(x.cuda(), qw, out_dtype=F32).double().cpu()
    ref = 30 * (x.double() @ D[N:].double().cpu().t())
    err, want, plain = ((h - ref).norm() / ref.norm()).item(), quotient(D[N:, 64:], bits, UNIT[bits]), quotient(D[N:, 64:], bits, 1.0)
    print(f"  off by {err:.3g}, expected {want:.3g}, at f = 1 {plain:.3g}")
    assert err <= 1.15 * want + 5e-7
    assert 1.15 * want + 5e-7 < plain
