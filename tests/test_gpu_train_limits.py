"""GPU test of the layer's backward at as many rows as a call takes: more workgroups than one launch holds.  Outer rows and those
around the border between launches against 64 bits, the adapters' gradients against sums in 64 bits; tolerances as of the
ordinary tests."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def test_layer_backward_of_2_to_27_rows():
    M, N, K, r, s = 2 ** 27, 8, 64, 16, 0.5
    print(f"linear_dropout_bwd M={M} N={N} K={K}", flush=True)
    gen = lambda i: torch.Generator(device="cuda").manual_seed(i)  # noqa: E731
    qw = qlr.quantize(torch.randn((N, K), generator=gen(1), device="cuda") * 0.05, 4)
    W = qlr.dequantize(qw, F32).double()
    A = (torch.randn((r, K), generator=gen(2), device="cuda") * 0.1).to(BF)
    B = (torch.randn((N, r), generator=gen(3), device="cuda") * 0.3).to(BF)
    x = torch.empty((M, K), dtype=BF, device="cuda").normal_(generator=gen(4))
    dy = torch.empty((M, N), dtype=BF, device="cuda").normal_(generator=gen(5))
    dx, dA, dB = qlr.linear_dropout_bwd(dy, x, qw, A, B, s)
    torch.cuda.synchronize()
    Ad, Bd = A.double(), B.double()
    half = M // 2
    for rows in (slice(0, 300), slice(half - 300, half + 300), slice(M - 300, M)):
        d = dy[rows].double()
        ref, S = d @ W + s * (d @ Bd) @ Ad, d.abs() @ W.abs() + s * (d.abs() @ Bd.abs()) @ Ad.abs()
        err, tol = (dx[rows].double() - ref).abs(), 5e-3 * S + 1e-5 + 2.0 ** -8 * ref.abs()
        assert (err <= tol).all(), (rows, (err / tol).max().item())
    sums = [torch.zeros(n, dtype=torch.float64, device="cuda") for n in ((r, K), (r, K), (N, r), (N, r))]
    for m in range(0, M, 2 ** 22):
        d, xs = dy[m:m + 2 ** 22].double(), x[m:m + 2 ** 22].double()
        sums[0] += s * (d @ Bd).t() @ xs
        sums[1] += s * (d.abs() @ Bd.abs()).t() @ xs.abs()
        sums[2] += s * d.t() @ (xs @ Ad.t())
        sums[3] += s * d.abs().t() @ (xs.abs() @ Ad.abs().t())
    for got, ref, S, what in ((dA, sums[0], sums[1], "dA"), (dB, sums[2], sums[3], "dB")):
        err, tol = (got.double() - ref).abs(), 1e-4 * S + 1e-6
        assert (err <= tol).all(), (what, (err / tol).max().item())
    del x, dy, dx
    torch.cuda.empty_cache()
