"""GPU tests of the calls of many rows, whose weight is dequantized once and whose last tiles may be split along the
contraction, against 64-bit references: the gated block, and the input gradients under adapter dropout.

Tolerances as of the smaller calls (the weight enters rounded to bf16 once here too): g and v 5e-3 S + 1e-5, S the sum of the
absolute values of the terms, h what these allow; dx 5e-3 S + 1e-5 of the layer and 1e-2 S + 1e-5 of the block (dg and dv are
rounded too); dA and dB 1e-4 S + 1e-6; and half a bf16 ulp for bf16 results."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402
from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import BF, F32, Train, close  # noqa: E402


def gated(L, act="silu", out=BF):
    h, gu = qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale, act, L.drop(), out_dtype=out, save=True)
    h2 = qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale, act, L.drop(), out_dtype=out)
    torch.cuda.synchronize()
    ref, tol, rgu, S = L.gated(act)
    close(gu, rgu, 5e-3 * S + 1e-5, "gu")
    close(h, ref, tol, "h")
    assert torch.equal(h, h2)


def gated_bwd(L, act="silu", out=BF):
    got = qlr.gated_bwd(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale, act, L.drop(), dx_dtype=out)
    torch.cuda.synchronize()
    (dx, Sx), a, b = L.gated_grads(act)
    close(got[0], dx, 1e-2 * Sx + 1e-5, "dx")
    if L.r:
        close(got[1], a[0], 1e-4 * a[1] + 1e-6, "dA")
        close(got[2], b[0], 1e-4 * b[1] + 1e-6, "dB")


def linear_bwd(L, out=BF):
    got = qlr.linear_dropout_bwd(L.dyd, L.xd, L.qw, L.Ad, L.Bd, L.scale, L.drop(), dx_dtype=out)
    torch.cuda.synchronize()
    (dx, Sx), a, b = L.grads(0, L.dy.double())
    close(got[0], dx, 5e-3 * Sx + 1e-5, "dx")
    if L.r:
        close(got[1], a[0], 1e-4 * a[1] + 1e-6, "dA")
        close(got[2], b[0], 1e-4 * b[1] + 1e-6, "dB")


@pytest.mark.parametrize("r", [0, 8])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_first(r, p):
    """One small call of each kind."""
    print(f"dense first r={r} p={p}", flush=True)
    L = Train(1024, 136, 192, 4, r, seed=1, sides=2, p=p)
    gated(L)
    gated_bwd(L)
    linear_bwd(Train(1024, 136, 192, 4, r, seed=1, p=p))


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("M", [1023, 1024, 1025, 1281])
def test_rows(bits, M):
    print(f"dense bits={bits} M={M}", flush=True)
    L = Train(M, 72, 192, bits, 8, seed=bits + M, sides=2, p=0.2)
    gated(L)
    gated_bwd(L)
    linear_bwd(Train(M, 72, 192, bits, 8, seed=bits + M, p=0.2))


# N of the last: 53 column tiles by 5 row tiles, 256 whole ones and 9 in four parts
@pytest.mark.parametrize("M,N,K", [(1024, 1, 64), (1025, 129, 64), (1100, 7, 128), (1300, 255, 2048), (1090, 130, 3136), (1030, 6664, 4096)])
@pytest.mark.parametrize("r", [0, 3, 40, 72])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_forward_shapes(M, N, K, r, out):
    if N > 1000 and r in (0, 3):
        pytest.skip("one of the wide ranks is enough at the largest size")
    print(f"dense fwd M={M} N={N} K={K} r={r}", flush=True)
    gated(Train(M, N, K, 4, r, seed=N + K + r, sides=2, p=0.1 if r else 0.0), out=out)


# contractions that end inside a step (N = 8, 72, 1032), of two to four parts (1032 on), and whole tiles beside parts (K = 13376)
@pytest.mark.parametrize("M,N,K", [(1024, 8, 64), (1057, 72, 320), (1100, 1032, 576), (1030, 2056, 256), (1030, 1032, 13376)])
@pytest.mark.parametrize("r", [0, 1, 40, 72])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_backward_shapes(M, N, K, r, p):
    if K > 10000 and r != 40:
        pytest.skip("one rank is enough at the largest size")
    if not r and p:
        pytest.skip("no adapter, no mask")
    for out in (BF, F32):
        print(f"dense bwd M={M} N={N} K={K} r={r} p={p} {out}", flush=True)
        gated_bwd(Train(M, N, K, 4, r, seed=N + K + r, sides=2, p=p), out=out)
        linear_bwd(Train(M, N, K, 4, r, seed=N + K + r, p=p), out=out)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
def test_activations(act):
    L = Train(1100, 104, 256, 4, 8, seed=3, sides=2, p=0.1)
    gated(L, act)
    gated_bwd(L, act)


def test_mask_itself():
    """With A = B = 1, x = 1 and dy = 1 the adapter's part of dx is the mask's factor, element for element."""
    M, K = 1030, 128
    L = Train(M, K, K, 4, K, seed=3, p=0.25)
    eye = torch.eye(K, dtype=BF).cuda()
    x = torch.ones((M, K), dtype=BF, device="cuda")
    dx = qlr.linear_dropout_bwd(x, x, L.qw, eye, eye, 1.0, L.drop(), dx_dtype=F32)[0]
    plain = qlr.linear_dropout_bwd(x, x, L.qw, dx_dtype=F32)[0]
    torch.cuda.synchronize()
    f = oracle.dropout_factors(M, K, 0.25, L.seed, L.counter)
    assert ((dx - plain).cpu().double() - torch.from_numpy(f)).abs().max() < 1e-4


def test_nonfinite_values_stay_where_they_enter():
    M = 1030
    L = Train(M, 64, 128, 4, 8, seed=6, sides=2)
    h0, g0 = qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale, save=True)
    c = qlr.gated_bwd(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale)
    rows = (torch.arange(M) != 1027).cuda()
    for bad in (float("inf"), float("-inf"), float("nan")):
        x = L.xd.clone()
        x[1027, 5] = bad
        h, gu = qlr.gated(x, L.qw, L.Ad, L.Bd, L.scale, save=True)
        assert torch.equal(h[rows], h0[rows]) and torch.equal(gu[rows], g0[rows]) and not torch.isfinite(gu[1027]).any()
        B = L.Bd.clone()
        B[1, 9, 3] = bad
        gu = qlr.gated(L.xd, L.qw, L.Ad, B, L.scale, save=True)[1]
        cols = (torch.arange(128) != 64 + 9).cuda()
        assert torch.equal(gu[:, cols], g0[:, cols]) and not torch.isfinite(gu[:, 73]).any()
        A = L.Ad.clone()
        A[0, 4, 7] = bad
        gu = qlr.gated(L.xd, L.qw, A, L.Bd, L.scale, save=True)[1]
        assert torch.equal(gu[:, 64:], g0[:, 64:])
        dy = L.dyd.clone()
        dy[1027, 10] = bad
        got = qlr.gated_bwd(dy, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale)
        cols = (torch.arange(64) != 10).cuda()
        assert torch.equal(got[0][rows], c[0][rows]) and not torch.isfinite(got[0][1027]).any()
        assert torch.equal(got[2][:, cols], c[2][:, cols])


def test_rows_and_outputs_behind_the_call_stay():
    L = Train(1029, 40, 128, 4, 8, seed=6, sides=2, p=0.1)

    def guarded(rows, cols, dtype):
        buf = torch.full((rows + 16, cols), 7.25, dtype=dtype, device="cuda")
        return buf, buf[8:8 + rows]

    hb, h = guarded(1029, 40, BF)
    gb, gu = guarded(1029, 80, BF)
    qlr.GatedCall(L.xd, L.qw, L.Ad, L.Bd, L.scale, dropout=L.drop(), out=h, gu=gu)()
    xb, dx = guarded(1029, 128, BF)
    dA, dB = torch.empty((2, 8, 128), device="cuda"), torch.empty((2, 40, 8), device="cuda")
    qlr.GatedBwdCall(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale, dropout=L.drop(), dx=dx, dA=dA, dB=dB)()
    torch.cuda.synchronize()
    for b in (hb, gb, xb):
        assert (b[:8] == 7.25).all() and (b[-8:] == 7.25).all()


def test_repeats_and_replays_bit_for_bit():
    L = Train(1100, 1032, 1024, 4, 64, seed=7, sides=2, p=0.1)
    h, gu = qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale, "silu", L.drop(), save=True)
    b = qlr.gated_bwd(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale, "silu", L.drop())
    outs = [torch.empty_like(t) for t in (h, gu, *b)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls = [qlr.GatedCall(L.xd, L.qw, L.Ad, L.Bd, L.scale, dropout=L.drop(), out=outs[0], gu=outs[1]),
                 qlr.GatedBwdCall(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale, dropout=L.drop(), dx=outs[2], dA=outs[3], dB=outs[4])]
        for call in calls:
            call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for call in calls:
                call()
    for _ in range(3):
        for t in outs:
            t.fill_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(outs, (h, gu, *b)))
