"""The 8-bit-integer and expert-grouped calls together, as a mixture-of-experts block uses them: a projection held in
8-bit integers (tokens quantized once, two linears of them), a router on the GPU, rows gathered by expert, the
experts' two coded linears with their adapters, the weighted sum back to the tokens; and the block's
adapter gradients.  Against the same block in 64 bits on the CPU, with the same routing.

The comparison is by relative 2-norm: each linear's weight enters rounded to bf16 and each result is rounded to bf16 (2^-9
of it in the mean square, five roundings on a path that the activation's slope below 1.1 does not amplify): 2e-2 covers four
times their sum."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402

BF = torch.bfloat16
D, F, E, R, TOP = 256, 384, 6, 8, 2
SCALE = 0.5


class Block:
    def __init__(self, T, seed):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.T = T
        self.x = n(T, D).to(BF)
        self.wp, self.wg = n(D, D) * D ** -0.5, n(E, D) * D ** -0.5
        self.up, self.down = n(E * F, D) * D ** -0.5, n(E * D, F) * F ** -0.5
        self.A1, self.B1 = (n(E, R, D) * D ** -0.5).to(BF), (n(E, F, R) * 0.3).to(BF)
        self.A2, self.B2 = (n(E, R, F) * F ** -0.5).to(BF), (n(E, D, R) * 0.3).to(BF)
        self.dz = n(T, D).to(BF)
        self.p8, self.g8 = qlr.quantize_i8(self.wp.cuda()), qlr.quantize_i8(self.wg.cuda())
        self.q1, self.q2 = qlr.quantize(self.up.cuda(), 4), qlr.quantize(self.down.cuda(), 4)
        self.d = {k: getattr(self, k).cuda() for k in ("x", "A1", "B1", "A2", "B2", "dz")}

    def run(self):
        """Forward and adapter gradients on the GPU; no value reaches the host."""
        d = self.d
        xq = qlr.quantize_i8(d["x"])
        h = qlr.linear_i8(None, self.p8, xq=xq)
        logits = qlr.linear_i8(None, self.g8, xq=xq, out_dtype=torch.float32)
        top, ids = torch.topk(torch.softmax(logits, 1), TOP, dim=1)
        order = torch.argsort(ids.reshape(-1), stable=True)
        offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"),
                             torch.cumsum((ids.reshape(-1)[None] == torch.arange(E, device="cuda")[:, None]).sum(1), 0)])
        offsets = offsets.to(torch.int32)
        token = order // TOP
        rows = h[token].contiguous()
        a = qlr.linear_grouped(rows, self.q1, offsets, d["A1"], d["B1"], SCALE)
        s = torch.nn.functional.silu(a.float())
        b = s.to(BF)
        o = qlr.linear_grouped(b, self.q2, offsets, d["A2"], d["B2"], SCALE)
        gate = top.reshape(-1)[order]
        z = torch.zeros((self.T, D), device="cuda").index_add_(0, token, o.float() * gate[:, None])
        do = (d["dz"].float()[token] * gate[:, None]).to(BF)
        db, dA2, dB2 = qlr.linear_grouped_bwd(do, b, self.q2, offsets, d["A2"], d["B2"], SCALE)
        sg = torch.sigmoid(a.float())
        da = (db.float() * sg * (1 + a.float() * (1 - sg))).to(BF)
        dr, dA1, dB1 = qlr.linear_grouped_bwd(da, rows, self.q1, offsets, d["A1"], d["B1"], SCALE)
        return dict(z=z, h=h, ids=ids, gate=top, dr=dr, dA1=dA1, dB1=dB1, dA2=dA2, dB2=dB2, order=order, offsets=offsets)

    def reference(self, ids, gate):
        """The block in 64 bits with the given routing."""
        dq = lambda q, n: qlr.dequantize(q, torch.float32).cpu().double().view(E, n, -1)  # noqa: E731
        W1, W2 = dq(self.q1, F), dq(self.q2, D)
        P = self.p8.q.cpu().double() * self.p8.scale.cpu().double()[:, None]
        xq = qlr.quantize_i8(self.d["x"])
        h = (xq.q.cpu().double() * xq.scale.cpu().double()[:, None]) @ P.t()
        leaves = {k: getattr(self, k).double().requires_grad_() for k in ("A1", "B1", "A2", "B2")}
        h = h.requires_grad_()
        z = torch.zeros((self.T, D), dtype=torch.float64)
        for e in range(E):
            w1 = W1[e] + SCALE * leaves["B1"][e] @ leaves["A1"][e]
            w2 = W2[e] + SCALE * leaves["B2"][e] @ leaves["A2"][e]
            w = (gate * (ids == e)).sum(1)
            z = z + w[:, None] * (torch.nn.functional.silu(h @ w1.t()) @ w2.t())
        (z * self.dz.double()).sum().backward()
        return z.detach(), h.detach(), h.grad, {k: v.grad for k, v in leaves.items()}


def rel(a, b):
    a = a.double().cpu()
    return ((a - b).norm() / b.norm()).item()


@pytest.mark.parametrize("T", [1, 5, 64, 777])
def test_block(T):
    B = Block(T, seed=T)
    out = B.run()
    torch.cuda.synchronize()
    ids, gate = out["ids"].cpu(), out["gate"].double().cpu()
    z, h, dh, grads = B.reference(ids, gate)
    assert rel(out["h"], h) < 2 ** -8
    assert rel(out["z"], z) < 2e-2
    for k in grads:
        assert rel(out["d" + k], grads[k]) < 2e-2, k
    # the rows' input gradients, summed back to the tokens
    got = torch.zeros((T, D), dtype=torch.float64)
    got.index_add_(0, (out["order"] // TOP).cpu(), out["dr"].double().cpu())
    assert rel(got, dh) < 2e-2
    cnt = np.bincount(ids.reshape(-1).numpy(), minlength=E)
    assert np.array_equal(np.diff(out["offsets"].cpu().numpy()), cnt)


def test_prepared_calls_replayed_from_a_graph():
    """The block's library calls captured once and replayed with other tokens and another routing, eager work
    between the replays."""
    T = 40
    B = Block(T, seed=3)
    n = T * TOP
    x = torch.zeros((T, D), dtype=BF, device="cuda")
    rows = torch.zeros((n, D), dtype=BF, device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        proj = qlr.LinearI8Call(x, B.p8)
        up = qlr.GroupedCall(rows, B.q1, offsets, B.d["A1"], B.d["B1"], SCALE, out=torch.zeros((n, F), dtype=BF, device="cuda"))
        down = qlr.GroupedCall(up.y, B.q2, offsets, B.d["A2"], B.d["B2"], SCALE, out=torch.zeros((n, D), dtype=BF, device="cuda"))
        back = qlr.GroupedBwdCall(down.y, up.y, B.q2, offsets, B.d["A2"], B.d["B2"], SCALE)

        def calls():
            proj(), up(), down(), back()

        calls()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            calls()
    rng = np.random.RandomState(0)
    for k in range(4):
        g = torch.Generator().manual_seed(100 + k)
        x.copy_(torch.randn((T, D), generator=g).to(BF))
        rows.copy_(torch.randn((n, D), generator=g).to(BF))
        cnt = rng.multinomial(n, np.ones(E) / E)
        offsets.copy_(torch.tensor(np.concatenate([[0], np.cumsum(cnt)]), dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (proj.y, up.y, down.y, back.dx, back.dA, back.dB)]
        want = [qlr.linear_i8(x, B.p8), qlr.linear_grouped(rows, B.q1, offsets, B.d["A1"], B.d["B1"], SCALE)]
        want.append(qlr.linear_grouped(want[1], B.q2, offsets, B.d["A2"], B.d["B2"], SCALE))
        want += qlr.linear_grouped_bwd(want[2], want[1], B.q2, offsets, B.d["A2"], B.d["B2"], SCALE)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k
