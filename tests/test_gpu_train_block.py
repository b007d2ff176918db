"""The gated block as a fine-tuning step uses it: gate and up projections with adapter dropout, the down projection with its own,
and all gradients; against the same block in 64 bits on the CPU, with the same masks.

By relative 2-norm: three linears' weights, the block's saved pre-activations, h, dh, dg and dv each rounded to bf16, 2^-9 of it in the
mean square, with |act'| below 1.13: 2e-2 covers four times the sum of the eight."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402
from quantized_base_fine_amd import qlr  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
D, F, R, SCALE, P, SEED = 256, 512, 16, 0.5, 0.1, 77


class Block:
    """Adapter masks: counters 3 c (gate), 3 c + 1 (up), 3 c + 2 (down) of step c."""

    def __init__(self, M, seed, act):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.M, self.act = M, act
        self.w1, self.w2 = qlr.quantize((n(2 * F, D) * D ** -0.5).cuda(), 4), qlr.quantize((n(D, F) * F ** -0.5).cuda(), 3)
        self.host = dict(x=n(M, D).to(BF), dz=n(M, D).to(BF), A1=(n(2, R, D) * D ** -0.5).to(BF), B1=(n(2, F, R) * 0.3).to(BF),
                         A2=(n(R, F) * F ** -0.5).to(BF), B2=(n(D, R) * 0.3).to(BF))
        self.d = {k: v.cuda() for k, v in self.host.items()}

    def calls(self, step):
        """Prepared forward and backward calls in the order of a step."""
        d, dr = self.d, lambda c: qlr.Dropout(P, SEED, c, step)  # noqa: E731
        up = qlr.GatedCall(d["x"], self.w1, d["A1"], d["B1"], SCALE, self.act, dr(0), save=True)
        down = qlr.LinearDropoutCall(up.h, self.w2, d["A2"], d["B2"], SCALE, dr(2))
        bdown = qlr.LinearDropoutBwdCall(d["dz"], up.h, self.w2, d["A2"], d["B2"], SCALE, dr(2))
        bup = qlr.GatedBwdCall(bdown.dx, up.gu, d["x"], self.w1, d["A1"], d["B1"], SCALE, self.act, dr(0))
        return up, down, bdown, bup

    def reference(self, c):
        """(z, gradients) in 64 bits by automatic differentiation."""
        w1, w2 = (qlr.dequantize(q, F32).cpu().double() for q in (self.w1, self.w2))
        leaf = {k: v.double().requires_grad_() for k, v in self.host.items() if k != "dz"}

        def lin(x, W, A, B, ctr):
            f = torch.from_numpy(oracle.dropout_factors(x.shape[0], x.shape[1], P, SEED, ctr))
            return x @ W.t() + SCALE * ((x * f) @ A.t()) @ B.t()

        g, v = (lin(leaf["x"], w1[i * F:(i + 1) * F], leaf["A1"][i], leaf["B1"][i], c + i) for i in (0, 1))
        a = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
             "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[self.act](g)
        z = lin(a * v, w2, leaf["A2"], leaf["B2"], c + 2)
        (z * self.host["dz"].double()).sum().backward()
        return z.detach(), {k: t.grad for k, t in leaf.items()}


def rel(a, b):
    return ((a.double().cpu() - b).norm() / b.norm()).item()


def check(B, calls, c):
    up, down, bdown, bup = calls
    z, grad = B.reference(c)
    assert rel(down.y, z) < 2e-2
    for k, t in (("x", bup.dx), ("A1", bup.dA), ("B1", bup.dB), ("A2", bdown.dA), ("B2", bdown.dB)):
        assert rel(t, grad[k]) < 2e-2, k


@pytest.mark.parametrize("M", [1, 16, 100, 700])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_step(M, act):
    B = Block(M, M, act)
    step = torch.tensor([12], dtype=torch.int64, device="cuda")
    calls = B.calls(step)
    for call in calls:
        call()
    torch.cuda.synchronize()
    check(B, calls, 12)


def test_captured_step():
    """The whole step captured once and replayed with the step's counter raised by three on the device, eager work between."""
    B = Block(70, 3, "silu")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls = B.calls(step)
        for call in calls:
            call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for call in calls:
                call()
    for k in range(3):
        step.fill_(3 * k)
        B.d["x"].copy_(torch.randn((70, D), generator=torch.Generator().manual_seed(50 + k)).to(BF))
        B.host["x"] = B.d["x"].cpu()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(B, calls, 3 * k)


def test_two_streams_at_once():
    """Calls with workspaces of their own on two streams together give what each gives alone."""
    Bs = [Block(300, 5 + i, "silu") for i in (0, 1)]
    step = torch.tensor([5], dtype=torch.int64, device="cuda")
    want = []
    for B in Bs:
        calls = B.calls(step)
        for call in calls:
            call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in (calls[0].h, calls[1].y, calls[2].dA, calls[2].dB, calls[3].dx, calls[3].dA, calls[3].dB)])
    streams = [torch.cuda.Stream() for _ in Bs]
    both = []
    for B, s in zip(Bs, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            both.append(B.calls(step))
    for _ in range(5):
        for i in range(4):
            for calls in both:
                calls[i]()
    torch.cuda.synchronize()
    for calls, w in zip(both, want):
        got = (calls[0].h, calls[1].y, calls[2].dA, calls[2].dB, calls[3].dx, calls[3].dA, calls[3].dB)
        assert all(torch.equal(a, b) for a, b in zip(got, w))


def test_gradients_against_differences():
    """The loss sum(z dz) along a random direction of all adapters, by central differences of the GPU's own forward in float32
    outputs.  The forward's rounding is the same bf16 weight on both sides of a difference, so what remains is h rounded to bf16:
    a relative 2^-8 on a difference of 1e-2 of the value, averaged over 70 x 256 terms, plus the gradients' own 2^-8: 5e-2."""
    B = Block(70, 4, "silu")
    B.d["x"] = (B.host["x"].float() * 0.5).to(BF).cuda()
    g = torch.Generator().manual_seed(9)
    base = {k: B.d[k].float() for k in ("A1", "B1", "A2", "B2")}
    way = {k: torch.randn(v.shape, generator=g).cuda() * v.abs().mean() for k, v in base.items()}
    dz = B.d["dz"].double()

    def loss(e):
        for k in base:
            B.d[k] = (base[k] + e * way[k]).to(BF)
        up, down, *_ = B.calls(None)
        up()
        y = qlr.linear_dropout(up.h, B.w2, B.d["A2"], B.d["B2"], SCALE, qlr.Dropout(P, SEED, 2), out_dtype=F32)
        return (y.double() * dz).sum().item(), {k: B.d[k].double() for k in base}

    (hi, ph), (lo, pl) = loss(0.25), loss(-0.25)
    for k in base:
        B.d[k] = ((ph[k] + pl[k]) / 2).to(BF)
    calls = B.calls(None)
    for call in calls:
        call()
    grad = dict(A1=calls[3].dA, B1=calls[3].dB, A2=calls[2].dA, B2=calls[2].dB)
    slope = sum((grad[k].double() * (ph[k] - pl[k])).sum().item() for k in base)
    size = sum((grad[k].double() * (ph[k] - pl[k])).norm().item() for k in base)
    assert abs((hi - lo) - slope) < 5e-2 * max(abs(slope), size), (hi - lo, slope)
