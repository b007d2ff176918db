"""GPU test of the gated block's gradients where the activation's slope is near its zero, act' = q + g q' with two terms that cancel:
against 64 bits, with the sizes of the two counted in S.  Each is off by less than 1e-6 (1 + w) of itself as the activation is (w its
exponent's size, below 2 here), so that the tolerances of the ordinary sizes hold (1e-4 S + 1e-6 for dA and dB, 1e-2 S + 1e-5 for dx)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402
from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import F32, Train, close  # noqa: E402

ACTS = ["silu", "gelu", "gelu_tanh"]

# the bf16 numbers next to the slopes' zeros
ZEROS = {"silu": [-1.28125, -1.2734375], "gelu": [-0.75, -0.75390625], "gelu_tanh": [-0.75, -0.75390625]}


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,r", [(1, 8, 8), (20, 64, 40), (600, 64, 8)])
def test_slope_near_its_zero(act, M, N, r):
    print(f"slope {act} M={M}", flush=True)
    for g0 in ZEROS[act]:
        L = Train(M, N, 128, 4, r, seed=M, sides=2)
        L.gu[:, :N] = g0
        L.gu[:, N:] *= 100
        L.gud = L.gu.cuda()
        got = qlr.gated_bwd(L.dyd, L.gud, L.xd, L.qw, L.Ad, L.Bd, L.scale, act, dx_dtype=F32)
        torch.cuda.synchronize()
        (dx, _), a, b = L.gated_grads(act)
        dh, g, v = L.dy.double(), L.gu[:, :N].double(), L.gu[:, N:].double()
        q, slope = (torch.from_numpy(t) for t in oracle.gate(g.numpy(), act))
        # act' = q + g q': the sum of the sizes of the two
        S = [L.grads(0, (dh * v).abs() * (q + (slope - q).abs())), L.grads(1, (dh * g * q).abs())]
        close(got[0], dx, 1e-2 * (S[0][0][1] + S[1][0][1]) + 1e-5, "dx")
        close(got[1], a[0], 1e-4 * torch.stack([S[0][1][1], S[1][1][1]]) + 1e-6, "dA")
        close(got[2], b[0], 1e-4 * torch.stack([S[0][2][1], S[1][2][1]]) + 1e-6, "dB")
