"""GPU test of the calls under adapter dropout and of the gated block with ranks past one tile of adapter columns, against 64-bit
references with the tolerances of the ordinary sizes (the scale falls with the rank, so that the adapter does not drown the base)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import Train, close  # noqa: E402


def layer(L):
    y = qlr.linear_dropout(L.xd, L.qw, L.Ad, L.Bd, L.scale, L.drop())
    got = qlr.linear_dropout_bwd(L.dyd, L.xd, L.qw, L.Ad, L.Bd, L.scale, L.drop())
    torch.cuda.synchronize()
    ref, S = L.linear(0)
    close(y, ref, 5e-3 * S + 1e-5, "y")
    check(got, *L.grads(0, L.dy.double()), 5e-3)


def block(L):
    h, gu = qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale, "gelu", L.drop(), save=True)
    got = qlr.gated_bwd(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale, "gelu", L.drop())
    torch.cuda.synchronize()
    ref, tol, rgu, S = L.gated("gelu")
    close(gu, rgu, 5e-3 * S + 1e-5, "gu")
    close(h, ref, tol, "h")
    check(got, *L.gated_grads("gelu"), 1e-2)


def check(got, dx, a, b, rel):
    close(got[0], dx[0], rel * dx[1] + 1e-5, "dx")
    close(got[1], a[0], 1e-4 * a[1] + 1e-6, "dA")
    close(got[2], b[0], 1e-4 * b[1] + 1e-6, "dB")


@pytest.mark.parametrize("M", [1, 3, 16, 40, 600])
@pytest.mark.parametrize("r", [65, 128, 300, 1024])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_rows(M, r, p):
    print(f"wide ranks M={M} r={r} p={p}", flush=True)
    for sides, run in ((1, layer), (2, block)):
        L = Train(M, 72, 320, 4, r, seed=M + r, sides=sides, p=p)
        L.scale = 16.0 / r
        run(L)


@pytest.mark.parametrize("r,p", [(136, 0.0), (136, 0.1), (200, 0.1)])
def test_many_rows(r, p):
    print(f"wide ranks, many rows r={r} p={p}", flush=True)
    L = Train(1537, 9400, 128, 4, r, seed=r, sides=2, p=p)
    L.scale = 16.0 / r
    h, gu = qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale, "silu", L.drop(), save=True)
    ref, tol, rgu, S = L.gated("silu")
    close(gu, rgu, 5e-3 * S + 1e-5, "gu")
    close(h, ref, tol, "h")
    for sides, N in ((1, 8200), (2, 4104)):
        L = Train(1537, N, 3648, 4, r, seed=r, sides=sides, p=p)
        L.scale = 16.0 / r
        if sides == 1:
            check(qlr.linear_dropout_bwd(L.dyd, L.xd, L.qw, L.Ad, L.Bd, L.scale, L.drop()), *L.grads(0, L.dy.double()), 5e-3)
        else:
            check(qlr.gated_bwd(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale, "silu", L.drop()), *L.gated_grads("silu"), 1e-2)
