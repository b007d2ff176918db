"""GPU tests of the layer under adapter dropout and of its gradients against 64-bit references.

Tolerances, per element, S the sum of the absolute values of the terms: y as the layer's families (1e-3 S + 1e-5 for the decode
kernels, 5e-3 S + 1e-5 for the tiled one, whose weight enters rounded to bf16, 2^-8 = 3.9e-3 of it); dx 5e-3 S + 1e-5 for the
same reason; dA and dB are float32 sums over products of at most 16 + 16 kept bits: 1e-4 S + 1e-6.  Half a bf16 ulp, 2^-8 of the value, is
added for bf16 results.  The kept elements' factor is one float32 rounding (6e-8) in every term."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402
from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import BF, F32, Train, close  # noqa: E402


def fwd(L, out=BF, path=qlr.PATH_AUTO):
    with qlr.path(path):
        y = qlr.linear_dropout(L.xd, L.qw, L.Ad, L.Bd, L.scale, L.drop(), out_dtype=out)
    torch.cuda.synchronize()
    ref, S = L.linear(0)
    rel = 5e-3 if path == qlr.PATH_GEMM or (path == qlr.PATH_AUTO and L.M > 16) else 1e-3
    close(y, ref, rel * S + 1e-5, "y")
    return y


def bwd(L, out=BF, need_dx=True):
    got = qlr.linear_dropout_bwd(L.dyd, L.xd, L.qw, L.Ad, L.Bd, L.scale, L.drop(), dx_dtype=out, need_dx=need_dx)
    torch.cuda.synchronize()
    (dx, Sx), a, b = L.grads(0, L.dy.double())
    if need_dx:
        close(got[0], dx, 5e-3 * Sx + 1e-5, "dx")
    if L.r:
        close(got[1], a[0], 1e-4 * a[1] + 1e-6, "dA")
        close(got[2], b[0], 1e-4 * b[1] + 1e-6, "dB")
    return got


@pytest.mark.parametrize("p", [0.0, 0.3])
def test_first(p):
    """One small call of each kind."""
    print(f"dropout first p={p}", flush=True)
    L = Train(40, 64, 128, 4, 8, seed=1, p=p)
    fwd(L)
    bwd(L)


def probe(M, K, p, **kw):
    """An adapter that copies: A the first r unit rows, B the identity, a weight of zeros' size: y shows the mask itself."""
    L = Train(M, K, K, 4, K, seed=3, p=p, **kw)
    eye = torch.eye(K, dtype=BF)
    L.A, L.B, L.Ad, L.Bd, L.scale = eye, eye, eye.cuda(), eye.cuda(), 1.0
    L.x = torch.ones((M, K), dtype=BF)
    L.xd = L.x.cuda()
    return L


@pytest.mark.parametrize("M", [1, 16, 33, 600])
def test_mask_itself(M):
    """With A = B = 1 and x = 1 the adapter's part is the mask's factor, element for element."""
    L = probe(M, 128, 0.25, counter=(1 << 40) + 5)
    base = qlr.linear(L.xd, L.qw, out_dtype=F32)
    y = qlr.linear_dropout(L.xd, L.qw, L.Ad, L.Bd, 1.0, L.drop(), out_dtype=F32)
    torch.cuda.synchronize()
    f = oracle.dropout_factors(M, 128, 0.25, L.seed, L.counter)
    assert ((y - base).cpu().double() - torch.from_numpy(f)).abs().max() < 1e-4
    # the same mask in the input gradient: dy = 1, u = 1, so dx - dy W' is the factor again
    L.dyd = torch.ones((M, 128), dtype=BF, device="cuda")
    dx = qlr.linear_dropout_bwd(L.dyd, L.xd, L.qw, L.Ad, L.Bd, 1.0, L.drop(), dx_dtype=F32)[0]
    plain = qlr.linear_dropout_bwd(L.dyd, L.xd, L.qw, dx_dtype=F32)[0]
    torch.cuda.synchronize()
    assert ((dx - plain).cpu().double() - torch.from_numpy(f)).abs().max() < 1e-4


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("M", [1, 5, 16, 17, 64, 65, 300])
def test_rows(bits, M):
    print(f"dropout bits={bits} M={M}", flush=True)
    L = Train(M, 72, 192, bits, 8, seed=bits + M, p=0.2)
    fwd(L)
    bwd(L)


@pytest.mark.parametrize("N,K", [(8, 64), (200, 320), (264, 512), (1032, 64), (96, 4096)])
@pytest.mark.parametrize("r", [1, 3, 16, 40, 72])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_shapes(N, K, r, out):
    print(f"dropout N={N} K={K} r={r}", flush=True)
    L = Train(37, N, K, 4, r, seed=N + K + r, p=0.1)
    fwd(L, out)
    bwd(L, out)


@pytest.mark.parametrize("path,M", [(qlr.PATH_GEMV, 1), (qlr.PATH_GEMV, 16), (qlr.PATH_GEMM, 5), (qlr.PATH_GEMM, 100)])
def test_families(path, M):
    fwd(Train(M, 100, 4096, 4, 16, seed=M, p=0.15), path=path)
    fwd(Train(M, 100, 256, 3, 5, seed=M, p=0.15), out=F32, path=path)


def test_float32_family():
    for M in (3, 50):
        L = Train(M, 40, 256, 4, 8, seed=M, p=0.4)
        with qlr.path(qlr.PATH_F32):
            y = qlr.linear_dropout(L.xd, L.qw, L.Ad, L.Bd, L.scale, L.drop(), out_dtype=F32)
        ref, S = L.linear(0)
        close(y, ref, 1e-4 * S + 1e-6, "y")


@pytest.mark.parametrize("M", [511, 512, 513, 1100])
def test_long_batches(M):
    """Rows past one gradient chunk and on its border; large tiles of the input gradient; no input gradient."""
    L = Train(M, 64, 256, 4, 20, seed=M, p=0.1)
    fwd(L)
    bwd(L)
    bwd(L, need_dx=False)


@pytest.mark.parametrize("M,K", [(3000, 4096), (2900, 4352)])
def test_large_tiles(M, K):
    """256 x 256 tiles of the input gradient: 192 of them, and one round with a rest that runs as 128 x 128 ones."""
    bwd(Train(M, 64, K, 4, 40, seed=9, p=0.1))


@pytest.mark.parametrize("p", [1e-6, 2.0 ** -16, 0.999, 0.9999999])
def test_extreme_probabilities(p):
    """Nothing dropped, one number of 65536, nearly all."""
    L = Train(70, 64, 512, 4, 8, seed=4, p=p)
    fwd(L, F32)
    bwd(L, F32)


def test_no_rows_and_no_adapter():
    L = Train(0, 64, 128, 4, 8, seed=1, p=0.5)
    y = qlr.linear_dropout(L.xd, L.qw, L.Ad, L.Bd, 1.0, L.drop())
    dx, dA, dB = qlr.linear_dropout_bwd(L.dyd, L.xd, L.qw, L.Ad, L.Bd, 1.0, L.drop())
    assert y.shape == (0, 64) and dx.shape == (0, 128) and not dA.any() and not dB.any()
    L = Train(30, 64, 128, 4, 0, seed=1, p=0.5)
    assert torch.equal(qlr.linear_dropout(L.xd, L.qw, dropout=L.drop()), qlr.linear(L.xd, L.qw))
    got = qlr.linear_dropout_bwd(L.dyd, None, L.qw, dropout=L.drop())
    (dx, Sx), _, _ = L.grads(0, L.dy.double())
    close(got[0], dx, 5e-3 * Sx + 1e-5, "dx")
    assert got[1] is None and got[2] is None


def test_without_dropout_equals_the_linear():
    L = Train(100, 64, 256, 4, 8, seed=2)
    for p in (None, qlr.Dropout(0.0, 1)):
        assert torch.equal(qlr.linear_dropout(L.xd, L.qw, L.Ad, L.Bd, L.scale, p), qlr.linear(L.xd, L.qw, L.Ad, L.Bd, L.scale))


def test_counter_and_step_add_modulo_2_64():
    L = Train(50, 64, 256, 4, 16, seed=5, p=0.3, counter=1000)
    a = qlr.linear_dropout(L.xd, L.qw, L.Ad, L.Bd, L.scale, qlr.Dropout(0.3, L.seed, 1000))
    for c, st in ((0, 1000), (1001, -1), ((1 << 64) - 5, 1005)):
        d = qlr.Dropout(0.3, L.seed, c, torch.tensor([st], dtype=torch.int64, device="cuda"))
        assert torch.equal(qlr.linear_dropout(L.xd, L.qw, L.Ad, L.Bd, L.scale, d), a), (c, st)
    for d in (qlr.Dropout(0.3, L.seed, 1001), qlr.Dropout(0.3, L.seed + 1, 1000), qlr.Dropout(0.3, L.seed ^ (1 << 40), 1000)):
        assert not torch.equal(qlr.linear_dropout(L.xd, L.qw, L.Ad, L.Bd, L.scale, d), a)


def test_dropped_elements_count_as_zero_whatever_they_hold():
    """A NaN or an infinity where every mask drops it reaches nothing but the base's products of its own row."""
    L = Train(20, 64, 128, 4, 8, seed=6, p=0.5)
    f = oracle.dropout_factors(20, 128, 0.5, L.seed, L.counter)
    m, k = [int(v[0]) for v in (f == 0).nonzero()]
    clean = qlr.linear_dropout_bwd(L.dyd, L.xd, L.qw, L.Ad, L.Bd, L.scale, L.drop())
    y0 = qlr.linear_dropout(L.xd, L.qw, L.Ad, L.Bd, L.scale, L.drop())
    x = L.xd.clone()
    for bad in (float("nan"), float("inf")):
        x[m, k] = bad
        got = qlr.linear_dropout_bwd(L.dyd, x, L.qw, L.Ad, L.Bd, L.scale, L.drop())
        assert all(torch.equal(a, b) for a, b in zip(got, clean))
        y = qlr.linear_dropout(x, L.qw, L.Ad, L.Bd, L.scale, L.drop())
        other = torch.arange(20) != m
        assert torch.equal(y[other.cuda()], y0[other.cuda()]) and not torch.isfinite(y[m]).any()


def test_captured_calls_follow_the_step():
    """Forward and backward captured once; every replay has the mask of the step that the device then holds."""
    L = Train(96, 64, 256, 4, 16, seed=8, p=0.2)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d = qlr.Dropout(0.2, L.seed, 3, step)
        f = qlr.LinearDropoutCall(L.xd, L.qw, L.Ad, L.Bd, L.scale, d)
        b = qlr.LinearDropoutBwdCall(L.dyd, L.xd, L.qw, L.Ad, L.Bd, L.scale, d)
        f(), b()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            f(), b()
    for k in (0, 4, 1 << 35, 4):
        step.fill_(k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (f.y, b.dx, b.dA, b.dB)]
        e = qlr.Dropout(0.2, L.seed, 3 + k)
        want = [qlr.linear_dropout(L.xd, L.qw, L.Ad, L.Bd, L.scale, e),
                *qlr.linear_dropout_bwd(L.dyd, L.xd, L.qw, L.Ad, L.Bd, L.scale, e)]
        assert all(torch.equal(a, c) for a, c in zip(got, want)), k


def test_repeats_bit_for_bit():
    L = Train(1100, 512, 1024, 4, 64, seed=7, p=0.1)
    a = qlr.linear_dropout_bwd(L.dyd, L.xd, L.qw, L.Ad, L.Bd, L.scale, L.drop())
    for _ in range(3):
        assert all(torch.equal(u, v) for u, v in
                   zip(a, qlr.linear_dropout_bwd(L.dyd, L.xd, L.qw, L.Ad, L.Bd, L.scale, L.drop())))


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("M", [17, 64, 65, 300])
@pytest.mark.parametrize("N,K", [(1, 512), (101, 1088), (255, 4096), (1032, 512)])
def test_ranges_of_the_contraction(bits, M, N, K):
    """The tiled product in two to eight ranges, odd widths, one step more in some."""
    print(f"dropout ranges bits={bits} M={M} N={N} K={K}", flush=True)
    L = Train(M, N, K, bits, 16 if bits == 4 else 5, seed=bits + M, p=0.1)
    fwd(L)
    fwd(L, F32)
