"""GPU tests of sizes whose workgroups number past what one launch holds (2^32 threads): outer rows, and those
around the borders between launches, against 64 bits.  Tolerances as in the ordinary tests of each call."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()  # (tens of GB)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def within(got, ref, S, rel, ab, what):
    tol = rel * S + ab + (2.0 ** -8 * ref.abs() if got.dtype == BF else 0)
    err = (got.double().cpu() - ref).abs()
    assert (err <= tol).all(), f"{what}: worst {(err / tol).max().item():.3g} of the tolerance"


def i8_slice(x, w8, sx, rows, cols):
    """(xq wq^T) sx sw of some rows and columns."""
    q = x[rows].double().cpu() * sx[rows].double().cpu()[:, None]
    return q @ (w8.q[cols].double().cpu() * w8.scale[cols].double().cpu()[:, None]).t()


def test_i8_few_rows_of_a_long_weight():
    M, N, K = 2, 2 ** 27 + 40, 16
    print(f"linear_i8 M={M} N={N} K={K}", flush=True)
    w8 = qlr.I8Rows.empty(N, K, "cuda")
    w8.q.random_(-127, 128, generator=gen(1))
    w8.scale.uniform_(0.5, 1, generator=gen(2))
    xq = qlr.I8Rows.empty(M, K, "cuda")
    xq.q.random_(-127, 128, generator=gen(3))
    xq.scale.uniform_(0.5, 1, generator=gen(4))
    y = qlr.linear_i8(None, w8, xq=xq, out_dtype=F32)
    torch.cuda.synchronize()
    half = 2 ** 26
    for cols in (slice(0, 300), slice(half - 300, half + 300), slice(2 ** 27 - 300, 2 ** 27), slice(N - 300, N)):
        ref = i8_slice(xq.q, w8, xq.scale, slice(0, M), cols)
        within(y[:, cols], ref, ref.abs(), 4e-7, 1e-30, f"columns {cols}")


@pytest.mark.parametrize("M,K,xdt", [(2 ** 20 + 3, 16, F32), (2 ** 20 + 3, 16, BF), (2 ** 25 + 5, 64, BF)],
                         ids=["f32", "bf16, 16 columns", "bf16, 64 columns"])
def test_i8_adapter_of_many_tokens(M, K, xdt):
    N, r, scale = 16, 64, 0.5
    print(f"linear_i8 M={M} N={N} K={K} r={r} {xdt}", flush=True)
    x = torch.empty((M, K), dtype=xdt, device="cuda").normal_(generator=gen(5))
    w8 = qlr.quantize_i8(torch.empty((N, K), device="cuda").normal_(generator=gen(6)))
    A = (torch.empty((r, K), device="cuda").normal_(generator=gen(7)) * K ** -0.5).to(BF)
    B = (torch.empty((N, r), device="cuda").normal_(generator=gen(8)) * 0.2).to(BF)
    xq = qlr.quantize_i8(x)
    y = qlr.linear_i8(x, w8, A, B, scale, xq=xq, out_dtype=F32)
    torch.cuda.synchronize()
    Ad, Bd = A.double().cpu(), B.double().cpu()
    rows = [slice(0, 300), slice(M - 300, M)] + [slice(M * i // 16 - 40, M * i // 16 + 40) for i in range(1, 16)]
    for s in rows:
        base = i8_slice(xq.q, w8, xq.scale, s, slice(0, N))
        xd = x[s].double().cpu()
        ref = base + scale * (xd @ Ad.t()) @ Bd.t()
        S = scale * (xd.abs() @ Ad.abs().t()) @ Bd.abs().t()
        within(y[s], ref, S + 4e-3 * (base.abs() + ref.abs()), 1e-4, 1e-30, f"rows {s}")


def test_grouped_products_of_many_tiles():
    """2048 experts of one row each on 8192 column tiles, on the tiled kernel, and their gradients."""
    E, N, K, r, scale = 2048, 2 ** 20, 64, 1, 0.5
    print(f"grouped {E} experts of {N} x {K}, one row each", flush=True)
    qw = qlr.QWeight.empty(E * N, K, 2, "cuda")
    qw.codes.random_(0, 256, generator=gen(9))
    qw.absmax_q8.random_(100, 256, generator=gen(10))
    qw.absmax_c.fill_(1e-3)
    A = (torch.empty((E, r, K), device="cuda").normal_(generator=gen(11)) * K ** -0.5).to(BF)
    B = torch.empty((E, N, r), dtype=BF, device="cuda").normal_(generator=gen(12))
    x = torch.empty((E, K), dtype=BF, device="cuda").normal_(generator=gen(13))
    dy = torch.empty((E, N), dtype=BF, device="cuda").normal_(generator=gen(14))
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    with qlr.path(qlr.PATH_GEMM):
        y = qlr.linear_grouped(x, qw, off, A, B, scale)
    dx, dA, dB = qlr.linear_grouped_bwd(dy, x, qw, off, A, B, scale, dx_dtype=F32)
    torch.cuda.synchronize()
    one = N * K // 64
    for e in (0, 1023, 1024, 2047):
        w = qlr.QWeight(2, N, K, qw.codes[e * N * K // 4:][:N * K // 4], qw.absmax_q8[e * one:][:one],
                        qw.absmax_c[e * one // 256:][:one // 256])
        W = qlr.dequantize(w, F32).cpu().double()
        xd, dd, Ad, Bd = x[e:e + 1].cpu().double(), dy[e:e + 1].cpu().double(), A[e].cpu().double(), B[e].cpu().double()
        t, u = xd @ Ad.t(), dd @ Bd
        ta, ua = xd.abs() @ Ad.abs().t(), dd.abs() @ Bd.abs()
        within(y[e:e + 1], xd @ W.t() + scale * t @ Bd.t(), xd.abs() @ W.abs().t() + scale * ta @ Bd.abs().t(), 5e-3, 1e-5, f"y {e}")
        within(dx[e:e + 1], dd @ W + scale * u @ Ad, dd.abs() @ W.abs() + scale * ua @ Ad.abs(), 5e-3, 1e-5, f"dx {e}")
        within(dA[e], scale * u.t() @ xd, scale * ua.t() @ xd.abs(), 1e-4, 1e-6, f"dA {e}")
        within(dB[e], scale * dd.t() @ t, scale * dd.abs().t() @ ta, 1e-4, 1e-6, f"dB {e}")


def test_grouped_backward_of_a_wide_adapter():
    """B transposed with 2^32 elements (a rank that is no multiple of 8)."""
    N, K, r, T, scale = 2 ** 20, 64, 4097, 3, 0.5
    print(f"grouped bwd {N} x {K} r={r}", flush=True)
    qw = qlr.QWeight.empty(N, K, 2, "cuda")
    qw.codes.random_(0, 256, generator=gen(15))
    qw.absmax_q8.random_(100, 256, generator=gen(16))
    qw.absmax_c.fill_(1e-3)
    A = (torch.empty((1, r, K), device="cuda").normal_(generator=gen(17)) * K ** -0.5).to(BF)
    B = torch.empty((1, N, r), dtype=BF, device="cuda").normal_(generator=gen(18))
    x = torch.empty((T, K), dtype=BF, device="cuda").normal_(generator=gen(19))
    dy = torch.empty((T, N), dtype=BF, device="cuda").normal_(generator=gen(20))
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    _, dA, _ = qlr.linear_grouped_bwd(dy, x, qw, off, A, B, scale, need_dx=False)
    torch.cuda.synchronize()
    xd, dd = x.cpu().double(), dy.cpu().double()
    for j in (0, 1, 2047, 4080, 4095, 4096):
        b = B[0, :, j].cpu().double()
        u, ua = dd @ b, dd.abs() @ b.abs()
        within(dA[0, j], scale * u @ xd, scale * ua @ xd.abs(), 1e-4, 1e-6, f"dA {j}")
