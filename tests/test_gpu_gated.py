"""GPU tests of the gated feed-forward block's first half and of its gradients against 64-bit references.

Tolerances, per element, S the sum of the absolute values of the terms: g and v 5e-3 S + 1e-5 (the weight enters rounded to
bf16, 2^-8 = 3.9e-3 of it), h what these allow through act(g) v (|act'| < 1.13); dx 1e-2 S + 1e-5 (the weight and dg, dv each
rounded to bf16: 2 x 3.9e-3); dA and dB 1e-4 S + 1e-6 (dg and dv in three bf16 parts, float32 sums).  Half a bf16 ulp, 2^-8 of
the value, is added for bf16 results."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import BF, F32, Train, close  # noqa: E402

ACTS = ["silu", "gelu", "gelu_tanh"]


def fwd(L, act="silu", out=BF, path=qlr.PATH_AUTO):
    with qlr.path(path):
        h, gu = qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale, act, L.drop(), out_dtype=out, save=True)
        h2 = qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale, act, L.drop(), out_dtype=out)
    torch.cuda.synchronize()
    ref, tol, rgu, S = L.gated(act)
    close(gu, rgu, 5e-3 * S + 1e-5, "gu")
    close(h, ref, tol, "h")
    assert torch.equal(h, h2)
    return h, gu


def bwd(L, act="silu", out=BF, need_dx=True):
    got = qlr.gated_bwd(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale, act, L.drop(), dx_dtype=out, need_dx=need_dx)
    torch.cuda.synchronize()
    (dx, Sx), a, b = L.gated_grads(act)
    if need_dx:
        close(got[0], dx, 1e-2 * Sx + 1e-5, "dx")
    if L.r:
        close(got[1], a[0], 1e-4 * a[1] + 1e-6, "dA")
        close(got[2], b[0], 1e-4 * b[1] + 1e-6, "dB")
    return got


@pytest.mark.parametrize("M", [3, 40])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_first(M, p):
    """One small call of each kind."""
    print(f"gated first M={M} p={p}", flush=True)
    L = Train(M, 72, 128, 4, 8, seed=1, sides=2, p=p)
    fwd(L)
    bwd(L)


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("M", [1, 5, 16, 17, 64, 65, 300])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_rows(bits, M, p):
    print(f"gated bits={bits} M={M} p={p}", flush=True)
    L = Train(M, 72, 192, bits, 8, seed=bits + M, sides=2, p=p)
    fwd(L)
    bwd(L)


@pytest.mark.parametrize("N,K", [(1, 64), (7, 128), (16, 64), (63, 192), (65, 320), (255, 64), (520, 1088), (96, 4096)])
@pytest.mark.parametrize("r", [0, 3, 16, 40, 72])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_forward_shapes(N, K, r, out):
    print(f"gated fwd N={N} K={K} r={r}", flush=True)
    for M in (2, 70):
        fwd(Train(M, N, K, 4, r, seed=N + K + r, sides=2, p=0.1 if r else 0.0), out=out)


@pytest.mark.parametrize("N,K", [(8, 64), (200, 320), (264, 512), (1032, 64), (96, 4096)])
@pytest.mark.parametrize("r", [0, 1, 3, 16, 40, 72])
@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_backward_shapes(N, K, r, p, out):
    print(f"gated bwd N={N} K={K} r={r} p={p}", flush=True)
    bwd(Train(37, N, K, 4, r, seed=N + K + r, sides=2, p=p if r else 0.0), out=out)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [4, 90])
def test_activations(act, M):
    L = Train(M, 104, 256, 4, 8, seed=3, sides=2, p=0.1)
    L.gu[:, 0], L.gu[:, 104] = 9.0, -3.0      # far out, where the slope is 1 or 0 almost
    L.gu[:, 1], L.gu[:, 2], L.gu[:, 3] = -12.0, 0.0, 88.0
    L.gud = L.gu.cuda()
    fwd(L, act)
    bwd(L, act)


def test_large_pre_activations():
    """Rows a hundred times as large: |g| to the thousands, where the exponential overflows on one side."""
    for act in ACTS:
        for M in (3, 33):
            L = Train(M, 64, 128, 4, 8, seed=5, sides=2, xscale=100.0)
            fwd(L, act, F32)
            L.gu = (L.gu * 100).to(BF)
            L.gud = L.gu.cuda()
            bwd(L, act)


@pytest.mark.parametrize("path,M", [(qlr.PATH_GEMV, 1), (qlr.PATH_GEMV, 16), (qlr.PATH_GEMM, 1), (qlr.PATH_GEMM, 16)])
def test_families(path, M):
    fwd(Train(M, 100, 4096, 4, 16, seed=M, sides=2, p=0.15), path=path)
    fwd(Train(M, 100, 256, 3, 5, seed=M, sides=2), out=F32, path=path)


@pytest.mark.parametrize("N", [5000, 16500, 33000])
def test_decode_widths(N):
    """One and two sets of rows to a workgroup."""
    for M in (1, 13):
        fwd(Train(M, N, 128, 4, 16, seed=N, sides=2))


@pytest.mark.parametrize("r", [64, 200])
def test_decode_wide_adapters(r):
    for M in (1, 16):
        fwd(Train(M, 80, 2048, 4, r, seed=r, sides=2))


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("M", [1500, 2048, 2500])
def test_large_tiles(bits, M):
    """Forward: 256 x 256 tiles of 128 columns, 32 of them by 6 to 10 row tiles (192, 256, and 320 with a rest of 64)."""
    fwd(Train(M, 4096, 64, bits, 8, seed=bits, sides=2, p=0.1))


@pytest.mark.parametrize("M,K", [(3000, 4096), (2900, 4352)])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_large_tiles_of_the_input_gradient(M, K, p):
    bwd(Train(M, 64, K, 4, 40, seed=9, sides=2, p=p))


@pytest.mark.parametrize("M", [511, 512, 513, 1100])
def test_long_batches(M):
    L = Train(M, 64, 256, 4, 20, seed=M, sides=2, p=0.1)
    fwd(L)
    bwd(L)
    bwd(L, need_dx=False)


def test_no_rows():
    L = Train(0, 64, 128, 4, 8, seed=1, sides=2, p=0.5)
    h, gu = qlr.gated(L.xd, L.qw, L.Ad, L.Bd, 1.0, "silu", L.drop(), save=True)
    dx, dA, dB = qlr.gated_bwd(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, 1.0, "silu", L.drop())
    assert h.shape == (0, 64) and gu.shape == (0, 128) and dx.shape == (0, 128) and not dA.any() and not dB.any()


def test_two_linears_under_dropout():
    """The gate's mask is that of a linear with the call's counter, the up projection's that of the next counter."""
    L = Train(50, 64, 256, 4, 16, seed=5, sides=2, p=0.3, counter=41, step=9)
    gu = qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale, "silu", L.drop(), save=True)[1]
    nb = 64 * 256 // 64
    # (copies: the buffers of a weight are 16-byte aligned)
    halves = [qlr.QWeight(4, 64, 256, L.qw.codes[i * nb * 32:(i + 1) * nb * 32].clone(),
                          L.qw.absmax_q8[i * nb:(i + 1) * nb].clone(), L.qw.absmax_c[i * nb // 256:].clone()) for i in (0, 1)]
    for i in (0, 1):
        d = qlr.Dropout(0.3, L.seed, 50 + i)
        y = qlr.linear_dropout(L.xd, halves[i], L.Ad[i].clone(), L.Bd[i].clone(), L.scale, d)
        ref, S = L.linear(i)
        for got in (y, gu[:, i * 64:(i + 1) * 64]):
            close(got, ref, 5e-3 * S + 1e-5, str(i))


def test_rows_and_outputs_behind_the_call_stay():
    """Outputs are views into larger buffers: what lies before and behind keeps its value."""
    L = Train(21, 40, 128, 4, 8, seed=6, sides=2, p=0.1)

    def guarded(rows, cols, dtype):
        buf = torch.full((rows + 16, cols), 7.25, dtype=dtype, device="cuda")
        return buf, buf[8:8 + rows]

    hb, h = guarded(21, 40, BF)
    gb, gu = guarded(21, 80, BF)
    qlr.GatedCall(L.xd, L.qw, L.Ad, L.Bd, L.scale, dropout=L.drop(), out=h, gu=gu)()
    xb, dx = guarded(21, 128, BF)
    ab, dA = guarded(16, 128, F32)
    bb, dB = guarded(80, 8, F32)
    qlr.GatedBwdCall(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale, dropout=L.drop(), dx=dx, dA=dA.view(2, 8, 128),
                     dB=dB.view(2, 40, 8))()
    torch.cuda.synchronize()
    for b in (hb, gb, xb, ab, bb):
        assert (b[:8] == 7.25).all() and (b[-8:] == 7.25).all()
    (rx, Sx), a, _ = L.gated_grads("silu")
    close(dx, rx, 1e-2 * Sx + 1e-5, "dx")
    close(dA.view(2, 8, 128), a[0], 1e-4 * a[1] + 1e-6, "dA")


@pytest.mark.parametrize("M", [8, 40])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_nonfinite_values_stay_where_they_enter(M, bad):
    """In x: its row.  In one adapter's A or B: that side of the columns it enters."""
    L = Train(M, 64, 128, 4, 8, seed=6, sides=2)
    h0, g0 = qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale, save=True)
    x = L.xd.clone()
    x[2, 5] = bad
    h, gu = qlr.gated(x, L.qw, L.Ad, L.Bd, L.scale, save=True)
    rows = (torch.arange(M) != 2).cuda()
    assert torch.equal(h[rows], h0[rows]) and torch.equal(gu[rows], g0[rows]) and not torch.isfinite(gu[2]).any()
    # the formula's signs where it has one: W' and the adapter's row times the infinity
    if bad != bad:
        return
    B = L.Bd.clone()
    B[1, 9, 3] = bad
    h, gu = qlr.gated(L.xd, L.qw, L.Ad, B, L.scale, save=True)
    cols = (torch.arange(128) != 64 + 9).cuda()
    assert torch.equal(gu[:, cols], g0[:, cols])
    t = (L.x.double() @ L.A[1].double().t())[:, 3]
    assert torch.equal(torch.sign(gu[:, 73].float()).cpu().double(), torch.sign(t * bad)) and torch.isinf(gu[:, 73]).all()
    A = L.Ad.clone()
    A[0, 4, 7] = bad
    h, gu = qlr.gated(L.xd, L.qw, A, L.Bd, L.scale, save=True)
    assert torch.equal(gu[:, 64:], g0[:, 64:])
    want = torch.sign(L.x[:, 7].double()[:, None] * bad * L.B[0, :, 4].double()[None])
    assert torch.equal(torch.sign(gu[:, :64].float()).cpu().double(), want) and torch.isinf(gu[:, :64]).all()


def test_backward_nonfinite():
    """An infinite upstream gradient: dx and dB of its row and column, dA through u; other columns of dB keep their values."""
    L = Train(20, 64, 128, 4, 8, seed=7, sides=2)
    c = qlr.gated_bwd(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale)
    dy = L.dyd.clone()
    dy[3, 10] = float("inf")
    got = qlr.gated_bwd(dy, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale)
    rows, cols = (torch.arange(20) != 3).cuda(), (torch.arange(64) != 10).cuda()
    assert torch.equal(got[0][rows], c[0][rows]) and not torch.isfinite(got[0][3]).any()
    assert torch.equal(got[2][:, cols], c[2][:, cols]) and torch.isinf(got[2][:, 10]).all()
    assert torch.isinf(got[1]).all()


def test_repeats_bit_for_bit():
    L = Train(1100, 512, 1024, 4, 64, seed=7, sides=2, p=0.1)
    f = qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale, "silu", L.drop(), save=True)
    b = qlr.gated_bwd(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale, "silu", L.drop())
    for _ in range(3):
        f2 = qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale, "silu", L.drop(), save=True)
        b2 = qlr.gated_bwd(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale, "silu", L.drop())
        assert all(torch.equal(u, v) for u, v in zip(f + b, f2 + b2))
