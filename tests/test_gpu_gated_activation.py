"""GPU test of the gated block's activations by themselves, against 64 bits.

Weights of zeros and ones give g and v exactly (g a bf16 number of x, v = 1), so that a float32 h is the activation and nothing
else.  Its bound, relative, with w the size of the exponent it takes (SiLU |g|, tanh GELU 2 c |g + 0.044715 g^3|, GELU g^2 / 2) and
u = 2^-24: the exponent is rounded once more than w (a product with log2 e, its constant to 1.4e-8): w (u + 1.4e-8) = 7.4e-8 w;
tanh GELU's w itself has six roundings, 3.6e-7 w; GELU's argument g / sqrt 2 has two, which erfc takes (2 x^2 + 1)-fold: 1.2e-7 (2 w
+ 1); exp2, the reciprocal (one ulp each), 1 + e and the product: 3.6e-7, erfc 2 ulp and two products.  Together under 1e-6 (1 + w); and below 2^-126 the
gate is 0: |g| 2^-126 < 2e-36 for |g| < 104, past which q is less still."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402
from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import BF, F32  # noqa: E402

ACTS = ["silu", "gelu", "gelu_tanh"]


def exponent(g, act):
    return {"silu": g.abs(), "gelu": g * g / 2, "gelu_tanh": 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3).abs()}[act]


def values():
    """bf16 numbers of both signs: over the whole range, and closely between 1/64 and 110."""
    m = torch.cat([torch.logspace(-30, 38, 160, dtype=torch.float64), torch.logspace(-6, math.log2(110), 608, base=2, dtype=torch.float64)])
    return torch.cat([m, -m]).to(BF)


def act_of(g, act, rows, N):
    """h of every g, `rows` rows to a call, through weights of zeros and ones (whole blocks of either: no level is 0, a scale is)."""
    W = torch.zeros((2 * N, 128))
    W[:N, :64], W[N:, 64:] = 1.0, 1.0
    qw = qlr.quantize(W.cuda(), 4)
    assert torch.equal(qlr.dequantize(qw, F32).cpu(), W)
    out = []
    for i in range(0, len(g), rows):
        x = torch.zeros((rows, 128), dtype=BF)
        n = min(rows, len(g) - i)
        x[:n, 0], x[:, 64] = g[i:i + n], 1.0
        h = qlr.gated(x.cuda(), qw, act=act, out_dtype=F32)
        assert torch.equal(h, h[:, :1].expand_as(h).contiguous())
        out.append(h[:n, 0].cpu())
    return torch.cat(out)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,N", [(16, 72), (64, 72), (1536, 11008)], ids=["decode", "tiles", "dense"])
def test_activation(act, rows, N):
    print(f"activation {act} rows={rows} N={N}", flush=True)
    g = values()
    got, gd = act_of(g, act, rows, N).double(), g.double()
    ref = gd * torch.from_numpy(oracle.gate(gd.numpy(), act)[0])
    err, w = (got - ref).abs(), exponent(gd, act)
    tol = 1e-6 * (1 + w) * ref.abs() + 2e-36
    worst = (err / tol).argmax()
    assert (err <= tol).all(), (g[worst].item(), got[worst].item(), ref[worst].item(), (err / tol)[worst].item())
