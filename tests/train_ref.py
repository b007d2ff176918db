"""64-bit references of the calls under adapter dropout and of the gated block, with the sums of absolute values that the
tolerances count (S of the header).  W' is the library's float32 dequantization (bit-exact against the oracle elsewhere);
masks and activations are the oracle's."""
import torch

import oracle
from quantized_base_fine_amd import qlr

BF, F32 = torch.bfloat16, torch.float32


class Train:
    """Inputs of one layer (sides = 1) or of a gated block (2), on the host in bfloat16 and on the GPU."""

    def __init__(self, M, N, K, bits, r, seed, sides=1, p=0.0, counter=7, step=None, xscale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.M, self.N, self.K, self.r, self.sides, self.p = M, N, K, r, sides, p
        self.qw = qlr.quantize((torch.randn((sides * N, K), generator=g) * 0.05).cuda(), bits)
        self.W = qlr.dequantize(self.qw, F32).double().view(sides, N, K)  # (the references' products run on the GPU in 64 bits)
        lead = (2,) if sides == 2 else ()
        self.x = (torch.randn((M, K), generator=g) * xscale).to(BF)
        self.A = (torch.randn((*lead, r, K), generator=g) * K ** -0.5).to(BF) if r else None
        self.B = (torch.randn((*lead, N, r), generator=g) * 0.2).to(BF) if r else None
        self.scale = 0.75 if r else 0.0
        self.dy = torch.randn((M, N), generator=g).to(BF)
        self.gu = (torch.randn((M, 2 * N), generator=g) * 2).to(BF)
        self.seed, self.counter, self.step = 0x1234567890ABCDEF + seed, counter, step
        self.xd, self.dyd, self.gud = self.x.cuda(), self.dy.cuda(), self.gu.cuda()
        self.Ad, self.Bd = (None, None) if not r else (self.A.cuda(), self.B.cuda())

    def drop(self):
        if self.p == 0.0:
            return None
        st = None if self.step is None else torch.tensor([self.step], dtype=torch.int64, device="cuda")
        return qlr.Dropout(self.p, self.seed, self.counter, st)

    def factors(self, side):
        return torch.from_numpy(oracle.dropout_factors(self.M, self.K, self.p, self.seed,
                                                       self.counter + side + (self.step or 0))).cuda()

    def ab(self, side):
        A, B = self.Ad.double(), self.Bd.double()
        return (A, B) if self.sides == 1 else (A[side], B[side])

    def linear(self, side):
        """(y, S) of one side."""
        x, W = self.x.double().cuda(), self.W[side]
        y, S = x @ W.t(), x.abs() @ W.abs().t()
        if self.r:
            (A, B), xk = self.ab(side), x * self.factors(side)
            y = y + self.scale * (xk @ A.t()) @ B.t()
            S = S + self.scale * (xk.abs() @ A.abs().t()) @ B.abs().t()
        return y.cpu(), S.cpu()

    def grads(self, side, dy):
        """((dx, S), (dA, S), (dB, S)) of one side for its upstream gradient."""
        x, W, s, dy = self.x.double().cuda(), self.W[side], self.scale, dy.cuda()
        dx, Sx = dy @ W, dy.abs() @ W.abs()
        if not self.r:
            return (dx.cpu(), Sx.cpu()), None, None
        (A, B), f = self.ab(side), self.factors(side)
        xk = x * f
        u, t, ua, ta = dy @ B, xk @ A.t(), dy.abs() @ B.abs(), xk.abs() @ A.abs().t()
        out = ((dx + s * f * (u @ A), Sx + s * f * (ua @ A.abs())), (s * u.t() @ xk, s * ua.t() @ xk.abs()),
               (s * dy.t() @ t, s * dy.abs().t() @ ta))
        return tuple((a.cpu(), b.cpu()) for a, b in out)

    def gated(self, act):
        """(h, tolerance of h without its own rounding, [g | v], S of them)."""
        (g, Sg), (v, Sv) = self.linear(0), self.linear(1)
        q, slope = (torch.from_numpy(a) for a in oracle.gate(g.numpy(), act))
        eg, ev = 5e-3 * Sg + 1e-5, 5e-3 * Sv + 1e-5
        # h = act(g) v at g + eg, v + ev: |act'| is at most 1.13 for all three, so act moves by at most 1.13 eg
        a = g * q
        return a * v, 1.13 * eg * (v.abs() + ev) + (a.abs() + 1e-6) * ev + 2e-6 * (a * v).abs(), torch.cat([g, v], 1), \
            torch.cat([Sg, Sv], 1)

    def gated_grads(self, act):
        g, v, dh = self.gu[:, :self.N].double(), self.gu[:, self.N:].double(), self.dy.double()
        d = [torch.from_numpy(a) for a in oracle.gated_backward(dh.numpy(), g.numpy(), v.numpy(), act)]
        parts = [self.grads(i, d[i]) for i in (0, 1)]
        dx = (parts[0][0][0] + parts[1][0][0], parts[0][0][1] + parts[1][0][1])
        if not self.r:
            return dx, None, None
        return dx, *[tuple(torch.stack([parts[0][k][i], parts[1][k][i]]) for i in (0, 1)) for k in (1, 2)]


def close(got, ref, tol, what):
    """Every finite element of ref within tol (+ half a bf16 ulp of a bf16 result)."""
    live = torch.isfinite(ref)
    if got.dtype == BF:
        tol = tol + 2.0 ** -8 * ref.abs()
    g = got.double().cpu()
    assert g.shape == ref.shape, what
    assert torch.isfinite(g[live]).all(), what
    err = (g - ref).abs()
    bad = (err > tol) & live
    assert not bad.any(), f"{what}: {int(bad.sum())} of {int(live.sum())} outside, worst {(err / tol)[live].max().item():.3g} of the tolerance"
    return float((err / tol)[live].max()) if live.any() else 0.0

