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


# Sizes: forward at least 1536 rows and two rounds of 256 tiles of 256 rows x 128 columns (7 x 74 here), backward a contraction of
# 8192 and 96 tiles of 256 x 256 (7 x 15).  These contractions end inside a step of 64.
GATED, LAYER = (4104, 3648), (8200, 3648)


@pytest.mark.parametrize("r", [0, 8])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_first(r, p):
    """One call of each kind."""
    print(f"dense first r={r} p={p}", flush=True)
    gated(Train(1537, 9400, 64, 4, r, seed=1, sides=2, p=p))
    gated_bwd(Train(1537, *GATED, 4, r, seed=1, sides=2, p=p))
    linear_bwd(Train(1537, *LAYER, 4, r, seed=1, p=p))


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("M", [1535, 1536, 1793])
def test_rows(bits, M):
    print(f"dense bits={bits} M={M}", flush=True)
    gated(Train(M, 10888, 64, bits, 8, seed=bits + M, sides=2, p=0.2))
    gated_bwd(Train(M, 4104, 4160, bits, 8, seed=bits + M, sides=2, p=0.2))
    linear_bwd(Train(M, 8200, 4160, bits, 8, seed=bits + M, p=0.2))


# an odd width, three steps; two parts of the last tiles' contraction
@pytest.mark.parametrize("M,N,K", [(1537, 9400, 64), (1600, 9473, 192), (1537, 9352, 2112)])
@pytest.mark.parametrize("r", [0, 3, 40, 72])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_forward_shapes(M, N, K, r, out):
    print(f"dense fwd M={M} N={N} K={K} r={r}", flush=True)
    gated(Train(M, N, K, 4, r, seed=N + K + r, sides=2, p=0.1 if r else 0.0), out=out)


@pytest.mark.parametrize("r", [0, 1, 40, 72])
@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_backward_shapes(r, p, out):
    print(f"dense bwd r={r} p={p}", flush=True)
    gated_bwd(Train(1537, *GATED, 4, r, seed=r, sides=2, p=p), out=out)
    linear_bwd(Train(1600, *LAYER, 4, r, seed=r, p=p), out=out)


@pytest.mark.parametrize("p", [0.0, 0.1])
def test_whole_tiles_and_parts(p):
    """38 x 7 tiles: 256 whole ones and 10 in four parts; and parts of two."""
    linear_bwd(Train(1537, 8200, 9536, 4, 40, seed=3, p=p), out=F32)
    gated_bwd(Train(1537, 4104, 9536, 4, 8, seed=3, sides=2, p=p))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
def test_activations(act):
    gated(Train(1537, 9400, 64, 4, 8, seed=3, sides=2, p=0.1), act)
    gated_bwd(Train(1537, *GATED, 4, 8, seed=3, sides=2, p=0.1), act)


@pytest.mark.parametrize("N,K,sides", [(*GATED, 2), (*LAYER, 1), (8200, 9536, 1)])
def test_mask_itself(N, K, sides):
    """What the adapters add to dx, with the mask: the product without them has the same sums, so that the difference is the
    adapters' part up to the float32 roundings of the sums (2^-24 of dx each) and of their 16-bit operands (2^-16 of S)."""
    L = Train(1537, N, K, 4, 40, seed=5, sides=sides, p=0.25)
    call = qlr.linear_dropout_bwd if sides == 1 else lambda dy, *a, **k: qlr.gated_bwd(dy, L.gud, *a, **k)
    args = {} if sides == 1 else {"act": "silu"}
    dx = call(L.dyd, L.xd, L.qw, L.Ad, L.Bd, L.scale, dropout=L.drop(), dx_dtype=F32, **args)[0]
    plain = call(L.dyd, None, L.qw, dx_dtype=F32, **args)[0]
    ref, tol = 0, 1e-6 * dx.abs().double().cpu()
    if sides == 1:
        ds = [L.dy.double()]
    else:
        ds = [torch.from_numpy(a) for a in oracle.gated_backward(L.dy.double().numpy(), L.gu[:, :N].double().numpy(),
                                                                 L.gu[:, N:].double().numpy(), "silu")]
    for i, d in enumerate(ds):
        A, B = L.ab(i)
        f, d = L.factors(i), d.cuda()
        ref = ref + (L.scale * f * ((d @ B) @ A)).cpu()
        tol = tol + 1e-4 * (L.scale * f * ((d.abs() @ B.abs()) @ A.abs())).cpu()
    close(dx.double() - plain.double(), ref, tol + 1e-6, "the adapters' part of dx")


def test_nonfinite_values_stay_where_they_enter():
    M, N, K = 1537, 9400, 128
    L = Train(M, N, K, 4, 8, seed=6, sides=2)
    g0 = qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale, save=True)[1]
    G = Train(M, *GATED, 4, 8, seed=6, sides=2)
    c = qlr.gated_bwd(G.dyd, G.gud, G.xd, G.qw, G.Ad, G.Bd, G.scale)
    rows = (torch.arange(M) != 1530).cuda()
    for bad in (float("inf"), float("-inf"), float("nan")):
        x = L.xd.clone()
        x[1530, 5] = bad
        gu = qlr.gated(x, L.qw, L.Ad, L.Bd, L.scale, save=True)[1]
        assert torch.equal(gu[rows], g0[rows]) and not torch.isfinite(gu[1530]).any()
        B = L.Bd.clone()
        B[1, 9, 3] = bad
        gu = qlr.gated(L.xd, L.qw, L.Ad, B, L.scale, save=True)[1]
        cols = (torch.arange(2 * N) != N + 9).cuda()
        assert torch.equal(gu[:, cols], g0[:, cols]) and not torch.isfinite(gu[:, N + 9]).any()
        A = L.Ad.clone()
        A[0, 4, 7] = bad
        gu = qlr.gated(L.xd, L.qw, A, L.Bd, L.scale, save=True)[1]
        assert torch.equal(gu[:, N:], g0[:, N:])
        dy = G.dyd.clone()
        dy[1530, 10] = bad
        got = qlr.gated_bwd(dy, G.gud, G.xd, G.qw, G.Ad, G.Bd, G.scale)
        cols = (torch.arange(GATED[0]) != 10).cuda()
        assert torch.equal(got[0][rows], c[0][rows]) and not torch.isfinite(got[0][1530]).any()
        assert torch.equal(got[2][:, cols], c[2][:, cols])


def test_rows_and_outputs_behind_the_call_stay():
    M, N, K = 1541, 9401, 64
    L = Train(M, N, K, 4, 8, seed=6, sides=2, p=0.1)
    G = Train(M, *GATED, 4, 8, seed=6, sides=2, p=0.1)

    def guarded(rows, cols, dtype):
        buf = torch.full((rows + 16, cols), 7.25, dtype=dtype, device="cuda")
        return buf, buf[8:8 + rows]

    hb, h = guarded(M, N, BF)
    gb, gu = guarded(M, 2 * N, BF)
    qlr.GatedCall(L.xd, L.qw, L.Ad, L.Bd, L.scale, dropout=L.drop(), out=h, gu=gu)()
    xb, dx = guarded(M, GATED[1], BF)
    dA, dB = torch.empty((2, 8, GATED[1]), device="cuda"), torch.empty((2, GATED[0], 8), device="cuda")
    qlr.GatedBwdCall(G.dyd, G.gud, G.xd, G.qw, G.Ad, G.Bd, G.scale, dropout=G.drop(), dx=dx, dA=dA, dB=dB)()
    torch.cuda.synchronize()
    for b in (hb, gb, xb):
        assert (b[:8] == 7.25).all() and (b[-8:] == 7.25).all()


def test_repeats_and_replays_bit_for_bit():
    L = Train(1537, 9400, 192, 4, 64, seed=7, sides=2, p=0.1)
    G = Train(1537, *GATED, 4, 64, seed=7, sides=2, p=0.1)
    h, gu = qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale, "silu", L.drop(), save=True)
    b = qlr.gated_bwd(G.dyd, G.gud, G.xd, G.qw, G.Ad, G.Bd, G.scale, "silu", G.drop())
    outs = [torch.empty_like(t) for t in (h, gu, *b)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls = [qlr.GatedCall(L.xd, L.qw, L.Ad, L.Bd, L.scale, dropout=L.drop(), out=outs[0], gu=outs[1]),
                 qlr.GatedBwdCall(G.dyd, G.gud, G.xd, G.qw, G.Ad, G.Bd, G.scale, dropout=G.drop(), dx=outs[2], dA=outs[3], dB=outs[4])]
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
