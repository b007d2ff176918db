"""GPU test of the gated block's backward at pre-activations over bf16's whole range, against 64-bit references: far out the
slope is 1 or 0 and g^3 passes float32's largest value.  dh is small and v large where g is far out, so that dg = dh v act'(g) and dv =
dh act(g) stay inside the range.  Tolerances as of the ordinary sizes (test_gpu_gated.py)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import BF, F32, Train, close  # noqa: E402

FAR = [1.1e13, 2e13, 1e15, 1e19, 1e20, 1e30, 3e38]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,r", [(14, 8), (33, 40), (600, 8)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_far_pre_activations(act, M, r, sign):
    print(f"gated bwd far {act} M={M} r={r} sign={sign}", flush=True)
    L = Train(M, 64, 128, 4, r, seed=M + r, sides=2)
    far = torch.tensor([FAR[i % len(FAR)] for i in range(64)], dtype=torch.float64)
    L.gu[:, :64] = (sign * far).to(BF)                      # every column far out, by its own power
    L.gu[:, 64:] = (L.gu[:, 64:].double() * 1e30).to(BF)
    L.dy = (L.dy.double() * 1e-30).to(BF)
    L.gu[::3, :64] = L.dy.new_tensor(sign * 0.5)            # and rows of ordinary ones beside them
    L.gud, L.dyd = L.gu.cuda(), L.dy.cuda()
    got = qlr.gated_bwd(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale, act, dx_dtype=F32)
    torch.cuda.synchronize()
    (dx, Sx), a, b = L.gated_grads(act)
    assert all(torch.isfinite(t).all() for t in (dx, a[0], b[0]))
    close(got[0], dx, 1e-2 * Sx + 1e-5, "dx")
    close(got[1], a[0], 1e-4 * a[1] + 1e-6, "dA")
    close(got[2], b[0], 1e-4 * b[1] + 1e-6, "dB")


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_nan_pre_activation(act):
    """A NaN still enters what its term enters, and nothing else."""
    L = Train(20, 64, 128, 4, 8, seed=7, sides=2)
    c = qlr.gated_bwd(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale, act)
    gu = L.gud.clone()
    gu[3, 10] = float("nan")
    got = qlr.gated_bwd(L.dyd, gu, L.xd, L.qw, L.Ad, L.Bd, L.scale, act)
    rows, cols = (torch.arange(20) != 3).cuda(), (torch.arange(64) != 10).cuda()
    assert torch.equal(got[0][rows], c[0][rows]) and torch.isnan(got[0][3]).all()
    assert torch.equal(got[2][:, cols], c[2][:, cols]) and torch.isnan(got[2][:, 10]).all() and torch.isnan(got[1]).all()
