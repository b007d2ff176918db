"""GPU tests of infinities and NaN in live rows and adapters of the expert-grouped products, their gradients and the
8-bit-integer linear.

The references are the definitions in 64 bits on the CPU, where an infinity meets the arithmetic of IEEE 754: an element
is infinite with the sign that the formula gives it, NaN where the formula does (Inf - Inf, 0 Inf), and finite
otherwise, whichever kernel family takes the row.  Finite elements keep the bounds of the ordinary tests: 5e-3 S + 1e-5 for
y and dx, 1e-4 S + 1e-6 for dA and dB, S the sum of the absolute values of the terms, plus half a bf16 step (2^-8)
of a bf16 result."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from test_gpu_grouped import F32, Layer  # noqa: E402
from test_gpu_i8 import make, ref_rows  # noqa: E402

INF, NAN = float("inf"), float("nan")


def same(got, ref, S, rel, ab, what, live=None):
    got = got.double().cpu()
    live = torch.ones_like(ref, dtype=torch.bool) if live is None else live
    fin, nan = torch.isfinite(ref), torch.isnan(ref)
    assert torch.isnan(got)[nan & live].all(), f"{what}: not NaN where the formula is"
    inf = torch.isinf(ref) & live
    bad = (got != ref) & inf
    assert not bad.any(), f"{what}: {int(bad.sum())} of {int(inf.sum())} infinities are {got[bad][:4].tolist()}"
    fin = fin & live
    assert ((got - ref).abs() <= rel * S + ab)[fin].all(), f"{what}: finite elements"
    return int(inf.sum())


def upload(L):
    L.xd, L.dyd, L.Ad, L.Bd = L.x.cuda(), L.dy.cuda(), L.A.cuda(), L.B.cuda()


def forward(L, path, what):
    with qlr.path(path):
        y = qlr.linear_grouped(L.xd, L.qw, L.offsets, L.Ad, L.Bd, L.scale, out_dtype=F32)
    torch.cuda.synchronize()
    ref, S = L.forward()
    return same(y, ref, S, 5e-3, 1e-5, what)


def backward(L):
    dx, dA, dB = qlr.linear_grouped_bwd(L.dyd, L.xd, L.qw, L.offsets, L.Ad, L.Bd, L.scale, dx_dtype=F32)
    torch.cuda.synchronize()
    (rx, Sx), (rA, SA), (rB, SB) = L.backward()
    return (same(dx, rx, Sx, 5e-3, 1e-5, "dx"), same(dA, rA, SA, 1e-4, 1e-6, "dA"),
            same(dB, rB, SB, 1e-4, 1e-6, "dB"))


# 9, 3 and 40 rows: the few-rows kernel and the tiles; 600 rows: the large tiles and a second chunk of the gradients
CASES = {"x": lambda L: L.x.__setitem__((4, 7), INF), "x nan": lambda L: L.x.__setitem__((4, 7), NAN),
         "A": lambda L: L.A.__setitem__((0, 0, 5), -INF), "B": lambda L: L.B.__setitem__((0, 6, 0), INF),
         "dy": lambda L: L.dy.__setitem__((4, 3), -INF)}


@pytest.mark.parametrize("path", [qlr.PATH_AUTO, qlr.PATH_GEMM], ids=["auto", "gemm"])
@pytest.mark.parametrize("r", [1, 8, 40])
@pytest.mark.parametrize("where", ["x", "x nan", "A", "B"])
@pytest.mark.parametrize("counts", [[9, 3, 40], [600, 2, 0]], ids=["short", "long"])
def test_forward(counts, where, r, path):
    print(f"grouped fwd, {where} not finite, counts={counts} r={r} path={path}", flush=True)
    L = Layer(counts, 72, 192, 4, r, seed=3 + r)
    CASES[where](L)
    upload(L)
    infs = forward(L, path, where)
    if where in ("A", "B"):
        assert infs >= counts[0]  # (the infinities of the other case can all be NaN)


@pytest.mark.parametrize("r", [1, 8, 40])
@pytest.mark.parametrize("where", ["x", "x nan", "A", "B", "dy"])
@pytest.mark.parametrize("counts", [[9, 3, 40], [600, 2, 0]], ids=["short", "long"])
def test_backward(counts, where, r):
    print(f"grouped bwd, {where} not finite, counts={counts} r={r}", flush=True)
    L = Layer(counts, 72, 192, 4, r, seed=5 + r)
    CASES[where](L)
    upload(L)
    infX, infA, infB = backward(L)
    # (an infinity in A or B meets rows of both signs in dB and dA: NaN in the formula too)
    assert {"x": infA and infB, "dy": infA and infB, "A": infX, "B": infX, "x nan": True}[where]


@pytest.mark.parametrize("path", [qlr.PATH_AUTO, qlr.PATH_GEMM], ids=["auto", "gemm"])
def test_largest_products(path):
    """s t between the largest bf16 value (3.3895e38) and the largest float32 value (3.4028e38), B near 1e-30: finite results."""
    L = Layer([9, 40], 24, 64, 4, 8, seed=4)
    L.x[:], L.A[:], L.scale = 0, 0, 3.4e38
    L.x[:, 3], L.A[:, :, 3] = 1, 1
    L.B = (L.B.float() * 1e-36).to(L.B.dtype)
    upload(L)
    assert forward(L, path, "y") == 0


def test_neighbours_keep_their_bits():
    """A row with a NaN changes no other row."""
    L = Layer([9, 3, 40], 72, 192, 4, 8, seed=6)
    ys = []
    for v in (None, NAN):
        if v is not None:
            L.xd[4, 7] = L.xd[30, 0] = v
        ys.append(qlr.linear_grouped(L.xd, L.qw, L.offsets, L.Ad, L.Bd, L.scale))
    torch.cuda.synchronize()
    keep = torch.ones(L.T, dtype=torch.bool, device="cuda")
    keep[4] = keep[30] = False
    assert torch.equal(ys[0][keep], ys[1][keep]) and torch.isnan(ys[1][~keep]).all()


@pytest.mark.parametrize("path,M", [(qlr.PATH_GEMV, 5), (qlr.PATH_GEMM, 5), (qlr.PATH_AUTO, 70)], ids=["gemv", "gemm", "auto"])
@pytest.mark.parametrize("where", ["A", "B", "scale"])
def test_linear_i8(where, path, M):
    """The adapter of the 8-bit linear: infinities in A and B, and s t past the largest bf16 value."""
    x, w, A, B = make(M, 48, 256, 8, seed=12)
    scale = 0.5
    if where == "A":
        A[2, 5] = INF
    elif where == "B":
        B[6, 0] = -INF
    else:
        x[:], A[:], scale = 0, 0, 3.4e38
        x[:, 3], A[:, 3] = 1, 1
        B = (B.float() * 1e-36).to(B.dtype)
    w8 = qlr.quantize_i8(w.cuda())
    with qlr.path(path):
        y = qlr.linear_i8(x.cuda(), w8, A.cuda(), B.cuda(), scale, out_dtype=F32)
    torch.cuda.synchronize()
    (xq, sx), (wq, sw) = ref_rows(x), ref_rows(w)
    ref = torch.from_numpy(xq * sx[:, None].astype("f8")) @ torch.from_numpy(wq * sw[:, None].astype("f8")).t()
    xd, Ad, Bd = x.double(), A.double(), B.double()
    t, ta = xd @ Ad.t(), xd.abs() @ Ad.abs().t()
    infs = same(y, ref + scale * t @ Bd.t(), ref.abs() + scale * ta @ Bd.abs().t(), 1e-4, 1e-30, where)
    assert infs == (0 if where == "scale" else M if where == "B" else infs) and (where != "A" or infs > 0)
