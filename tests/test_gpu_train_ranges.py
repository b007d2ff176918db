"""GPU tests of split contractions where a row's sums are rounded up to four columns: gated blocks and layers of odd widths in
several ranges, against 64-bit references with the tolerances of the ordinary sizes, and with guards around the outputs."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import BF, F32, Train, close  # noqa: E402

ROWS = [17, 64, 65, 130]


def guarded(rows, cols, dtype):
    buf = torch.full((rows + 16, cols), 7.25, dtype=dtype, device="cuda")
    return buf, buf[8:8 + rows]


def untouched(*bufs):
    assert all((b[:8] == 7.25).all() and (b[-8:] == 7.25).all() for b in bufs)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("N", [1, 2, 3, 97, 130, 259])
@pytest.mark.parametrize("r,p", [(0, 0.0), (5, 0.2), (40, 0.0)])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_block(M, N, r, p, out):
    print(f"ranges block M={M} N={N} r={r} p={p}", flush=True)
    K = 2112 if N == 97 else 1024
    assert qlr.workspace_bytes(qlr.OP_GATED, M, N, K, 0) >= 2 * M * 2 * N * 4  # two ranges at least
    L = Train(M, N, K, 4, r, seed=M + N + r, sides=2, p=p)
    (hb, h), (gb, gu) = guarded(M, N, out), guarded(M, 2 * N, BF)
    qlr.GatedCall(L.xd, L.qw, L.Ad, L.Bd, L.scale, dropout=L.drop(), out=h, gu=gu)()
    torch.cuda.synchronize()
    ref, tol, rgu, S = L.gated("silu")
    close(gu, rgu, 5e-3 * S + 1e-5, "gu")
    close(h, ref, tol, "h")
    untouched(gb, hb)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("N", [1, 2, 3, 97, 130, 259])
@pytest.mark.parametrize("r", [5, 40])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_layer(M, N, r, out):
    print(f"ranges layer M={M} N={N} r={r}", flush=True)
    L = Train(M, N, 1088, 4, r, seed=M + N + r, p=0.2)
    yb, y = guarded(M, N, out)
    qlr.LinearDropoutCall(L.xd, L.qw, L.Ad, L.Bd, L.scale, dropout=L.drop(), out=y)()
    torch.cuda.synchronize()
    ref, S = L.linear(0)
    close(y, ref, 5e-3 * S + 1e-5, "y")
    untouched(yb)
