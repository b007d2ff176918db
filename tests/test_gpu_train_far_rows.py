"""GPU tests of masks of the largest inputs: groups of eight elements past 2^32 (rows of 2^20 columns), and as many rows as a call takes,
whose masked adapter products are more workgroups than one launch holds.  Chosen rows (outer ones and those around the border)
against 64 bits with the oracle's masks; everything else is zero where a sum runs over all rows.  Tolerances as of the ordinary sizes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402
from quantized_base_fine_amd import qlr  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
SEED, COUNTER, P, SCALE = 0xFEDCBA9876543210, 5, 0.3, 0.75


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()  # (tens of GB)


def factors(rows, K, counter):
    """(len(rows), K) float64 on the GPU: the oracle's mask and factor of chosen rows."""
    t, lo = oracle.dropout_threshold(P), np.uint64(0xFFFFFFFF)
    g = (np.asarray(rows, dtype=np.uint64)[:, None] * np.uint64(K // 8) + np.arange(K // 8, dtype=np.uint64)).reshape(-1)
    words = oracle.philox4x32((g & lo, g >> np.uint64(32), counter, 0), (SEED & 0xFFFFFFFF, SEED >> 32))
    n = np.stack([h for w in np.broadcast_arrays(*words) for h in (w & 0xFFFF, w >> 16)], 1)
    return torch.from_numpy(np.where(n >= t, 65536.0 / (65536 - t), 0.0).reshape(len(rows), K)).cuda()


def test_the_rows_factors_are_the_oracles():
    assert torch.equal(factors(range(5, 9), 64, COUNTER).cpu(), torch.from_numpy(oracle.dropout_factors(9, 64, P, SEED, COUNTER)[5:]))


def within(got, ref, tol, what):
    if got.dtype == BF:
        tol = tol + 2.0 ** -8 * ref.abs()
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), f"{what}: worst {(err / tol).max().item():.3g} of the tolerance"


class Rows:
    """A layer (sides = 1) or a gated block (2) of M rows, whose chosen rows have upstream gradients; columns: how many elements
    of a chosen row of x are not zero (None: all, of every row)."""

    def __init__(self, M, N, K, r, sides, rows, columns, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.rows, self.K, self.N, self.sides = rows, K, N, sides
        at = self.at = torch.tensor(rows, device="cuda")
        self.qw = qlr.quantize(normal(sides * N, K) * 0.05, 4)
        self.W = qlr.dequantize(self.qw, F32).double().view(sides, N, K)
        lead = (2,) if sides == 2 else ()
        self.A, self.B = (normal(*lead, r, K) * 0.2).to(BF), (normal(*lead, N, r) * 0.5).to(BF)
        if columns is None:
            self.x = torch.empty((M, K), dtype=BF, device="cuda").normal_(generator=gen)
        else:
            self.x = torch.zeros((M, K), dtype=BF, device="cuda")
            for m in rows:
                self.x[m, torch.randint(K, (columns,), generator=gen, device="cuda")] = normal(columns).to(BF)
        self.dy = torch.zeros((M, N), dtype=BF, device="cuda")
        self.dy[at] = normal(len(rows), N).to(BF)
        self.f = [factors(rows, K, COUNTER + i) for i in range(sides)]
        self.drop = qlr.Dropout(P, SEED, COUNTER)
        self.gen = gen

    def ab(self, i):
        return (self.A.double(), self.B.double()) if self.sides == 1 else (self.A[i].double(), self.B[i].double())

    def linear(self, i):
        x, (A, B), f = self.x[self.at].double(), self.ab(i), self.f[i]
        y = x @ self.W[i].t() + SCALE * ((x * f) @ A.t()) @ B.t()
        return y, x.abs() @ self.W[i].abs().t() + SCALE * ((x * f).abs() @ A.abs().t()) @ B.abs().t()

    def grads(self, i, d):
        x, (A, B), f, W = self.x[self.at].double(), self.ab(i), self.f[i], self.W[i]

        def of(x, d, W, A, B):
            xk = x * f
            return d @ W + SCALE * f * ((d @ B) @ A), SCALE * (d @ B).t() @ xk, SCALE * d.t() @ (xk @ A.t())

        return of(x, d, W, A, B), of(x.abs(), d.abs(), W.abs(), A.abs(), B.abs())

    def check_layer(self):
        print("layer forward", flush=True)
        y = qlr.linear_dropout(self.x, self.qw, self.A, self.B, SCALE, self.drop, out_dtype=F32)
        torch.cuda.synchronize()
        ref, S = self.linear(0)
        within(y[self.at], ref, 5e-3 * S + 1e-5, "y")
        print("layer backward", flush=True)
        dx, dA, dB = qlr.linear_dropout_bwd(self.dy, self.x, self.qw, self.A, self.B, SCALE, self.drop)
        torch.cuda.synchronize()
        (rx, ra, rb), (sx, sa, sb) = self.grads(0, self.dy[self.at].double())
        within(dx[self.at], rx, 5e-3 * sx + 1e-5, "dx")
        within(dA, ra, 1e-4 * sa + 1e-6, "dA")
        within(dB, rb, 1e-4 * sb + 1e-6, "dB")

    def check_block(self):
        print("block forward", flush=True)
        N = self.N
        h, gu = qlr.gated(self.x, self.qw, self.A, self.B, SCALE, "silu", self.drop, save=True)
        torch.cuda.synchronize()
        for i in (0, 1):
            ref, S = self.linear(i)
            within(gu[self.at, i * N:(i + 1) * N], ref, 5e-3 * S + 1e-5, f"side {i}")
        del h
        print("block backward", flush=True)
        dx, dA, dB = qlr.gated_bwd(self.dy, gu, self.x, self.qw, self.A, self.B, SCALE, "silu", self.drop)
        torch.cuda.synchronize()
        g, v = gu[self.at, :N].double().cpu().numpy(), gu[self.at, N:].double().cpu().numpy()
        ds = [torch.from_numpy(d).cuda() for d in oracle.gated_backward(self.dy[self.at].double().cpu().numpy(), g, v, "silu")]
        (r0, s0), (r1, s1) = self.grads(0, ds[0]), self.grads(1, ds[1])
        within(dx[self.at], r0[0] + r1[0], 1e-2 * (s0[0] + s1[0]) + 1e-5, "dx")
        for i, (r, s) in enumerate(((r0, s0), (r1, s1))):
            within(dA[i], r[1], 1e-4 * s[1] + 1e-6, f"dA {i}")
            within(dB[i], r[2], 1e-4 * s[2] + 1e-6, f"dB {i}")


# rows of 2^17 groups: from row 2^15 on a group's number takes 33 bits
M_FAR = 2 ** 15 + 16
FAR = [0, 3, 2 ** 15 - 2, 2 ** 15 - 1, 2 ** 15, 2 ** 15 + 1, M_FAR - 2, M_FAR - 1]


@pytest.mark.parametrize("sides", [1, 2])
def test_groups_past_32_bits(sides):
    print(f"groups past 2^32, sides={sides}", flush=True)
    L = Rows(M_FAR, 8, 2 ** 20, 8, sides, FAR, 64, seed=sides)
    assert all(not torch.equal(L.f[0][i], L.f[0][i + 4]) for i in range(2))
    L.check_layer() if sides == 1 else L.check_block()


def test_block_of_2_to_27_rows():
    """The two masked products: 2^22 row tiles of 32 rows each, in launches of 2^21."""
    M = 2 ** 27
    print(f"block of {M} rows", flush=True)
    rows = [*range(40), *range(M // 2 - 40, M // 2 + 40), *range(M - 40, M)]
    Rows(M, 8, 64, 8, 2, rows, None, seed=3).check_block()
