"""GPU tests of the expert-grouped products and their gradients against 64-bit references.

W' is the library's float32 dequantization (bit-exact against the oracle elsewhere); the references are float64 products per
expert on the CPU.  Tolerances, per element, with S the sum of the absolute values of the terms: the weight enters
rounded to bf16 (half a step, 2^-8 = 3.9e-3 of it) and float32 sums of at most a few hundred MFMA steps (below 1e-4 S):
5e-3 S + 1e-5 for y and dx, plus 2^-8 |y| for a bf16 result; dA and dB are float32 sums of exactly widened
inputs, u and t float32: 1e-4 S + 1e-6."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


class Layer:
    def __init__(self, counts, N, K, bits, r, seed, pad=0, lead=0):
        g = torch.Generator().manual_seed(seed)
        self.E, self.N, self.K, self.r = len(counts), N, K, r
        self.off = lead + np.concatenate([[0], np.cumsum(counts)])
        self.T = int(self.off[-1]) + pad
        self.qw = qlr.quantize((torch.randn((self.E * N, K), generator=g) * 0.05).cuda(), bits)
        self.W = qlr.dequantize(self.qw, F32).cpu().double().view(self.E, N, K)
        self.x = torch.randn((self.T, K), generator=g).to(BF)
        self.dy = torch.randn((self.T, N), generator=g).to(BF)
        self.A = (torch.randn((self.E, r, K), generator=g) * K ** -0.5).to(BF) if r else None
        self.B = (torch.randn((self.E, N, r), generator=g) * 0.2).to(BF) if r else None
        self.scale = 0.75 if r else 0.0
        # rows of no expert hold NaN: they must not be read
        for t in (self.x, self.dy):
            t[:lead] = float("nan")
            t[int(self.off[-1]):] = float("nan")
        self.offsets = torch.tensor(self.off, dtype=torch.int32, device="cuda")
        self.xd, self.dyd = self.x.cuda(), self.dy.cuda()
        self.Ad, self.Bd = (None, None) if not r else (self.A.cuda(), self.B.cuda())

    def rows(self):
        for e in range(self.E):
            a, b = int(self.off[e]), int(self.off[e + 1])
            if b > a:
                yield e, a, b

    def forward(self):
        """(y, S) with NaN in the rows of no expert."""
        y = torch.full((self.T, self.N), float("nan"), dtype=torch.float64)
        S = torch.zeros_like(y)
        for e, a, b in self.rows():
            x, W = self.x[a:b].double(), self.W[e]
            y[a:b], S[a:b] = x @ W.t(), x.abs() @ W.abs().t()
            if self.r:
                A, B = self.A[e].double(), self.B[e].double()
                y[a:b] += self.scale * (x @ A.t()) @ B.t()
                S[a:b] += self.scale * (x.abs() @ A.abs().t()) @ B.abs().t()
        return y, S

    def backward(self):
        dx = torch.full((self.T, self.K), float("nan"), dtype=torch.float64)
        Sx = torch.zeros_like(dx)
        dA, SA = [torch.zeros((self.E, self.r, self.K), dtype=torch.float64) for _ in range(2)]
        dB, SB = [torch.zeros((self.E, self.N, self.r), dtype=torch.float64) for _ in range(2)]
        for e, a, b in self.rows():
            x, dy, W = self.x[a:b].double(), self.dy[a:b].double(), self.W[e]
            dx[a:b], Sx[a:b] = dy @ W, dy.abs() @ W.abs()
            if self.r:
                A, B, s = self.A[e].double(), self.B[e].double(), self.scale
                u, t = dy @ B, x @ A.t()
                ua, ta = dy.abs() @ B.abs(), x.abs() @ A.abs().t()
                dx[a:b] += s * u @ A
                Sx[a:b] += s * ua @ A.abs()
                dA[e], SA[e] = s * u.t() @ x, s * ua.t() @ x.abs()
                dB[e], SB[e] = s * dy.t() @ t, s * dy.abs().t() @ ta
        return (dx, Sx), (dA, SA), (dB, SB)


def close(got, ref, S, rel, ab, what):
    live = torch.isfinite(ref)
    tol = rel * S + ab
    if got.dtype == BF:
        tol = tol + 2.0 ** -8 * ref.abs()
    g = got.double().cpu()
    assert torch.isfinite(g[live]).all(), what
    err = (g - ref).abs()
    bad = (err > tol) & live
    assert not bad.any(), f"{what}: {int(bad.sum())} of {int(live.sum())} outside, worst {(err / tol)[live].max().item():.3g} of the tolerance"


def check_forward(L, path="auto", out=BF):
    y0 = torch.full((L.T, L.N), 7.25, dtype=out, device="cuda")
    with qlr.path({"auto": qlr.PATH_AUTO, "gemm": qlr.PATH_GEMM}[path]):
        y = qlr.linear_grouped(L.xd, L.qw, L.offsets, L.Ad, L.Bd, L.scale, out=y0)
    torch.cuda.synchronize()
    ref, S = L.forward()
    close(y, ref, S, 5e-3, 1e-5, "y")
    assert (y.cpu()[~torch.isfinite(ref)] == 7.25).all(), "rows of no expert"
    return y


def check_backward(L, out=BF, need_dx=True):
    dx0 = torch.full((L.T, L.K), 7.25, dtype=out, device="cuda") if need_dx else None
    dx, dA, dB = qlr.GroupedBwdCall(L.dyd, L.xd, L.qw, L.offsets, L.Ad, L.Bd, L.scale, dx=dx0, need_dx=need_dx)()
    torch.cuda.synchronize()
    (rx, Sx), (rA, SA), (rB, SB) = L.backward()
    if need_dx:
        close(dx, rx, Sx, 5e-3, 1e-5, "dx")
        assert (dx.cpu()[~torch.isfinite(rx)] == 7.25).all(), "rows of no expert"
    else:
        assert dx is None
    if L.r:
        close(dA, rA, SA, 1e-4, 1e-6, "dA")
        close(dB, rB, SB, 1e-4, 1e-6, "dB")
        assert (dA[SA.sum((1, 2)) == 0] == 0).all() and (dB[SB.sum((1, 2)) == 0] == 0).all()
    return dx, dA, dB


COUNTS = [[1], [0, 1, 0], [16, 17, 15], [0, 0, 0], [300, 0, 5, 64], [1, 2, 3, 4, 5, 6, 7], [256, 257, 255], [40, 0, 16, 128, 33]]


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("path", ["auto", "gemm"])
def test_forward_counts(bits, counts, path):
    print(f"grouped fwd bits={bits} counts={counts} {path}", flush=True)
    check_forward(Layer(counts, 72, 192, bits, 8, seed=sum(counts) + bits, pad=3, lead=2), path)


@pytest.mark.parametrize("N,K", [(1, 64), (7, 128), (16, 64), (255, 320), (257, 64), (520, 1088), (96, 4096)])
@pytest.mark.parametrize("r", [0, 3, 16, 40, 72])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_forward_shapes(N, K, r, out):
    print(f"grouped fwd N={N} K={K} r={r}", flush=True)
    check_forward(Layer([3, 0, 70, 16], N, K, 4, r, seed=N + K + r, pad=2), out=out)


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
def test_backward_counts(bits, counts):
    print(f"grouped bwd bits={bits} counts={counts}", flush=True)
    check_backward(Layer(counts, 72, 192, bits, 8, seed=sum(counts) + bits, pad=3, lead=2))


@pytest.mark.parametrize("N,K", [(8, 64), (64, 128), (200, 320), (264, 512), (1032, 64)])
@pytest.mark.parametrize("r", [0, 3, 16, 72])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_backward_shapes(N, K, r, out):
    print(f"grouped bwd N={N} K={K} r={r}", flush=True)
    check_backward(Layer([3, 0, 70, 16], N, K, 4, r, seed=N + K + r, pad=2), out=out)


def test_backward_long_experts_and_no_input_gradient():
    """Experts past one gradient chunk (512 rows), on its border and one past it."""
    L = Layer([513, 512, 1, 1100], 48, 64, 4, 12, seed=5)
    check_backward(L)
    check_backward(L, need_dx=False)


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
def test_large_tiles_and_their_rest(bits):
    """Enough rows and columns for the 256 x 256 tiles: 64 column tiles, 11, 13 and 9 row tiles, so a last round of 192 tiles
    (kept whole), of 64 and of 64 (run as smaller tiles); the input gradient with 32 column tiles, 11 row tiles, 352 = 256 + 96."""
    for counts in ([500, 700, 256, 3, 1000], [520, 700, 256, 3, 1100], [512, 300, 1, 513, 200]):
        L = Layer(counts, 16384, 64, bits, 8, seed=sum(counts) + bits)
        check_forward(L)
    L = Layer([500, 0, 400, 900, 700], 64, 8192, bits, 8, seed=bits)
    check_backward(L)


@pytest.mark.parametrize("r", [8, 24, 64, 72])
def test_wide_adapters_and_half_filled_tiles(r):
    """Input gradient: 32 column tiles, 12 row tiles of 256, of which four hold at most 128 rows, 384 = 256 + 128 of them; the
    adapter products of ranges of 1 to 700 rows in steps of 32 and 64 rows."""
    L = Layer([384, 90, 300, 530, 1, 700], 64, 8192, 4, r, seed=r)
    check_backward(L)
    check_forward(L)


@pytest.mark.parametrize("counts", [[350] * 8, [350] * 7 + [600], [250] * 8 + [750]], ids=["16", "17", "11"])
@pytest.mark.parametrize("bits", [3, 4])
def test_about_one_round_of_large_tiles(bits, counts):
    """Input gradient: 16 column tiles of 256 and 16, 17 and 11 row tiles, so a whole round, one and 16 tiles, part of one."""
    check_backward(Layer(counts, 64, 4096, bits, 16, seed=sum(counts) + bits, pad=1))


def test_no_rows():
    L = Layer([0, 0], 24, 128, 4, 8, seed=1)
    assert qlr.linear_grouped(L.xd, L.qw, L.offsets, L.Ad, L.Bd, 1.0).shape == (0, 24)
    dx, dA, dB = qlr.linear_grouped_bwd(L.dyd, L.xd, L.qw, L.offsets, L.Ad, L.Bd, 1.0)
    torch.cuda.synchronize()
    assert dx.shape == (0, 128) and (dA == 0).all() and (dB == 0).all()


def test_offsets_out_of_range_or_decreasing_stay_inside_the_buffers():
    """The kernels clamp every offset into [0, T] and to its predecessor: guard rows around y and dx keep their values."""
    L = Layer([30, 40, 20], 40, 128, 4, 8, seed=2)
    for bad in ([0, 200, -5, 90], [-7, 10, 1 << 30, 50], [90, 60, 30, 0], [0, 90, 0, 90]):
        L.offsets.copy_(torch.tensor(bad, dtype=torch.int32))
        y = torch.full((L.T + 64, L.N), 7.25, dtype=BF, device="cuda")
        dx = torch.full((L.T + 64, L.K), 7.25, dtype=BF, device="cuda")
        qlr.linear_grouped(L.xd, L.qw, L.offsets, L.Ad, L.Bd, 1.0, out=y[32:32 + L.T])
        qlr.GroupedBwdCall(L.dyd, L.xd, L.qw, L.offsets, L.Ad, L.Bd, 1.0, dx=dx[32:32 + L.T])()
        torch.cuda.synchronize()
        for t in (y, dx):
            assert (t[:32] == 7.25).all() and (t[32 + L.T:] == 7.25).all()


def test_rows_and_codes_past_32_bit_offsets():
    """x past 2^32 bytes and codes past 2^32 bytes: the last expert's rows against 64 bits."""
    K, N, T = 2048, 64, 1_100_000
    g = torch.Generator(device="cuda").manual_seed(3)
    W = torch.randn((3 * N, K), generator=g, device="cuda") * 0.05
    qw = qlr.quantize(W, 4)
    x = torch.empty((T, K), dtype=BF, device="cuda")
    x.normal_(generator=g)
    assert x.numel() * 2 > 1 << 32
    for last in (9, 400_000):
        off = torch.tensor([0, 5, T - last, T], dtype=torch.int32, device="cuda")
        y = qlr.linear_grouped(x, qw, off)
        w = qlr.dequantize(qw, F32).view(3, N, K)
        for e, rows in ((2, slice(T - 9, T)), (1, slice(T - last - 300, T - last)), (0, slice(0, 5))):
            xr = x[rows].cpu().double()
            we = w[e].cpu().double()
            close(y[rows], xr @ we.t(), xr.abs() @ we.abs().t(), 5e-3, 1e-5, f"rows of expert {e}")
    del x, y
    E, N, K = 70, 8192, 8192
    qw = qlr.QWeight.empty(E * N, K, 8, "cuda")
    assert qw.codes.numel() > 1 << 32
    qw.codes.random_(0, 256, generator=g)
    qw.absmax_q8.random_(100, 256, generator=g)
    qw.absmax_c.fill_(1e-3)
    one = N * K // 64
    last = qlr.QWeight(8, N, K, qw.codes[(E - 1) * N * K:], qw.absmax_q8[(E - 1) * one:], qw.absmax_c[(E - 1) * one // 256:])
    w = qlr.dequantize(last, F32).cpu().double()
    for rows in (3, 90):
        x = torch.randn((rows, K), generator=g, device="cuda").to(BF)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[E] = rows
        y = qlr.linear_grouped(x, qw, off, out_dtype=F32)
        xr = x.cpu().double()
        close(y, xr @ w.t(), xr.abs() @ w.abs().t(), 5e-3, 1e-5, "last expert")
        dy = torch.randn((rows, N), generator=g, device="cuda").to(BF)
        dx, _, _ = qlr.linear_grouped_bwd(dy, None, qw, off, dx_dtype=F32)
        d = dy.cpu().double()
        close(dx, d @ w, d.abs() @ w.abs(), 5e-3, 1e-5, "last expert's input gradient")


def test_calls_on_two_streams():
    """Two calls in flight on two streams, each with a workspace of its own."""
    Ls = [Layer([50, 200, 9], 128, 512, 4, 16, seed=s) for s in (20, 21)]
    torch.cuda.synchronize()
    outs = []
    for L in Ls:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            outs.append([(qlr.linear_grouped(L.xd, L.qw, L.offsets, L.Ad, L.Bd, L.scale),
                          *qlr.linear_grouped_bwd(L.dyd, L.xd, L.qw, L.offsets, L.Ad, L.Bd, L.scale)) for _ in range(5)])
    torch.cuda.synchronize()
    for L, o in zip(Ls, outs):
        ref, S = L.forward()
        (rx, Sx), (rA, SA), (rB, SB) = L.backward()
        for y, dx, dA, dB in o:
            close(y, ref, S, 5e-3, 1e-5, "y")
            close(dx, rx, Sx, 5e-3, 1e-5, "dx")
            close(dA, rA, SA, 1e-4, 1e-6, "dA")
            close(dB, rB, SB, 1e-4, 1e-6, "dB")


def test_many_long_experts():
    """More experts than a wave has lanes, on large tiles and their rest: 70 ranges of 1 to 520 rows, 8 column tiles."""
    counts = [1 + (97 * i * i + 31 * i) % 520 for i in range(70)]
    assert sum(counts) >= 96 * 70
    L = Layer(counts, 2048, 64, 4, 8, seed=11, pad=2, lead=3)
    check_forward(L)
    L = Layer(counts, 64, 2048, 4, 8, seed=12)
    check_backward(L)


def test_many_experts():
    rng = np.random.RandomState(3)
    counts = rng.randint(0, 4, size=150)
    counts[70] = 40
    L = Layer(list(counts), 24, 64, 4, 4, seed=6, pad=1)
    check_forward(L)
    check_forward(L, "gemm")
    check_backward(L)


def test_results_do_not_depend_on_the_neighbours():
    """An expert's rows alone give the bits that they give among others (the same kernel family)."""
    L = Layer([40, 9, 33], 80, 256, 4, 8, seed=8)
    with qlr.path(qlr.PATH_GEMM):
        y = qlr.linear_grouped(L.xd, L.qw, L.offsets, L.Ad, L.Bd, L.scale)
        one = torch.tensor([0, 0, 9, 9], dtype=torch.int32, device="cuda")
        z = qlr.linear_grouped(L.xd[40:49].contiguous(), L.qw, one, L.Ad, L.Bd, L.scale)
    torch.cuda.synchronize()
    assert torch.equal(y[40:49], z)


def test_repeated_calls_give_the_same_bits():
    L = Layer([700, 3, 90], 96, 320, 4, 16, seed=10)
    a = [t.clone() for t in (qlr.linear_grouped(L.xd, L.qw, L.offsets, L.Ad, L.Bd, L.scale),
                             *qlr.linear_grouped_bwd(L.dyd, L.xd, L.qw, L.offsets, L.Ad, L.Bd, L.scale))]
    for _ in range(3):
        b = (qlr.linear_grouped(L.xd, L.qw, L.offsets, L.Ad, L.Bd, L.scale),
             *qlr.linear_grouped_bwd(L.dyd, L.xd, L.qw, L.offsets, L.Ad, L.Bd, L.scale))
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_captured_call_follows_the_offsets():
    """Offsets are read on the GPU: a captured forward and backward replayed with other offsets."""
    L = Layer([20, 4, 40], 64, 128, 4, 8, seed=12)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = torch.zeros((L.T, L.N), dtype=BF, device="cuda")
    dx = torch.zeros((L.T, L.K), dtype=BF, device="cuda")
    with torch.cuda.stream(side):
        f = qlr.GroupedCall(L.xd, L.qw, L.offsets, L.Ad, L.Bd, L.scale, out=y)
        b = qlr.GroupedBwdCall(L.dyd, L.xd, L.qw, L.offsets, L.Ad, L.Bd, L.scale, dx=dx)
        f(), b()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            f(), b()
    for counts in ([20, 4, 40], [0, 64, 0], [1, 1, 1], [33, 30, 1], [0, 0, 0]):
        L.off = np.concatenate([[0], np.cumsum(counts)])
        L.offsets.copy_(torch.tensor(L.off, dtype=torch.int32))
        y.fill_(0), dx.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref, S = L.forward()
        close(y, ref, S, 5e-3, 1e-5, f"y {counts}")
        (rx, Sx), (rA, SA), (rB, SB) = L.backward()
        close(dx, rx, Sx, 5e-3, 1e-5, f"dx {counts}")
        close(b.dA, rA, SA, 1e-4, 1e-6, f"dA {counts}")
        close(b.dB, rB, SB, 1e-4, 1e-6, f"dB {counts}")
        assert (y.cpu()[~torch.isfinite(ref)] == 0).all() and (dx.cpu()[~torch.isfinite(rx)] == 0).all()


def test_gradients_against_differences():
    """dA, dB and dx of a loss sum(y * dy) against central differences of the reference forward in 64 bits."""
    L = Layer([5, 0, 3], 16, 64, 8, 4, seed=14)
    dx, dA, dB = check_backward(L, out=F32)
    rng = np.random.RandomState(0)

    def loss():
        y, _ = L.forward()
        return float((torch.nan_to_num(y) * L.dy.double()).sum())

    L.x, L.A, L.B = L.x.double(), L.A.double(), L.B.double()
    for t, g in ((L.x, dx), (L.A, dA), (L.B, dB)):
        flat, grad = t.view(-1), g.double().cpu().view(-1)
        for i in rng.randint(0, flat.numel(), size=12):
            h, v = 1e-3, flat[i].item()
            flat[i] = v + h
            up = loss()
            flat[i] = v - h
            down = loss()
            flat[i] = v
            # the loss is at most quadratic in one element: the difference is exact up to float64 rounding; dx
            # carries the bf16 weights (checked above against S), so it is compared with its scale
            d = (up - down) / (2 * h)
            assert abs(d - grad[i].item()) <= 2e-2 * max(1.0, abs(d)), (i, d, grad[i].item())
