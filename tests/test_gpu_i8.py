"""GPU tests of the 8-bit-integer linear layer: row quantization (exact), the product on both
kernel families, the adapter, scales of non-finite and zero rows.

The reference is numpy / torch on the CPU in 64 bits, from the definitions: s = fl32(max|x| fl32(1 / 127)), q the integer
nearest x / s (ties to even), y = sx sw sum(xq wq) + scale (x A^T) B^T.

Tolerance of the product: the integer sum is exact; its conversion and the two scale products round three
times and the adapter's sum once (2^-24 each, so 4 * 2^-24 < 4e-7 of the base and of the result); the adapter's term keeps
16 significant bits of t (2^-16) and float32 sums of at most K / 64 + 64 partial steps: 1e-4 of its magnitude
sum covers both; a bf16 result is off by half a step, 2^-8 of it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def ref_rows(x):
    """(q float64, scale float32) of a CPU tensor by the definition, in 64 bits."""
    v = x.float().numpy()
    bad = ~np.isfinite(v).all(1)
    am = np.where(bad, 0.0, np.abs(np.where(np.isfinite(v), v, 0)).max(1)).astype(np.float32)
    s = (am * (np.float32(1) / np.float32(127))).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        q = np.rint(v.astype(np.float64) / s.astype(np.float64)[:, None])
    q = np.clip(np.where((s > 0)[:, None] & ~bad[:, None], q, 0), -127, 127)
    return q, np.where(bad, np.float32(np.nan), s)


def rand(rows, cols, seed, dt="bf16", scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, cols), generator=g) * scale).to(DT[dt])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 64), (2, 2048), (17, 4096), (3, 16384), (2, 16392), (2, 20001),
                                       (300, 136)])
def test_quantize_rows_exact(rows, cols, dt):
    print(f"quantize_i8 {rows}x{cols} {dt}", flush=True)
    x = rand(rows, cols, rows * 31 + cols, dt, 3.0)
    q = qlr.quantize_i8(x.cuda())
    torch.cuda.synchronize()
    rq, rs = ref_rows(x)
    assert np.array_equal(q.scale.cpu().numpy(), rs)
    assert np.array_equal(q.q.cpu().numpy().astype(np.float64), rq)


def test_quantize_ties_go_to_even_and_borders_keep_their_side():
    # absmax 127 gives scale 1: every half-integer is a tie; its float32 neighbours are not
    h = np.arange(-126.5, 127, 1.0, dtype=np.float32)
    row = np.concatenate([h, np.nextafter(h, np.float32(200)), np.nextafter(h, np.float32(-200)), [127.0, -127.0]])
    x = torch.from_numpy(np.stack([row, row * np.float32(0.37), row * np.float32(2.0 ** -120), row * np.float32(1e30)])
                         .astype(np.float32))
    q = qlr.quantize_i8(x.cuda())
    rq, rs = ref_rows(x)
    assert np.array_equal(q.scale.cpu().numpy(), rs)
    assert np.array_equal(q.q.cpu().numpy().astype(np.float64), rq)
    assert q.q[0, 0].item() == -126 and q.q[0, 126].item() == 0  # -126.5 -> -126, -0.5 -> 0


def test_quantize_agrees_with_torch_on_the_gpu():
    """The same scales and integers as amax() / 127 and a division on the GPU (short rows: many exact ties)."""
    x = rand(2000, 264, 9).cuda()
    q = qlr.quantize_i8(x)
    s = x.float().abs().amax(1) / 127
    assert torch.equal(q.scale, s)
    assert torch.equal(q.q.double(), torch.round(x.double() / s.double()[:, None]).clamp(-127, 127))


def test_quantize_more_rows_than_one_launch_holds():
    x = torch.randn((2 ** 23 + 5, 16), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).to(torch.bfloat16)
    q = qlr.quantize_i8(x)
    torch.cuda.synchronize()
    for a, b in ((0, 300), (2 ** 23 - 100, 2 ** 23 + 5)):
        rq, rs = ref_rows(x[a:b].cpu())
        assert np.array_equal(q.scale[a:b].cpu().numpy(), rs)
        assert np.array_equal(q.q[a:b].cpu().numpy().astype(np.float64), rq)
    assert torch.equal(q.scale, x.float().abs().amax(1) / 127)


def test_quantize_extreme_rows():
    x = torch.zeros((8, 72), dtype=torch.float32)
    x[1, 5] = float("nan")
    x[2, 6] = float("inf")
    x[3, 0] = -float("inf")
    x[4] = torch.linspace(-1, 1, 72) * 3.4e38
    x[5] = torch.linspace(-1, 1, 72) * 1e-38
    x[6] = torch.arange(72) * 2.0 ** -149
    x[7, 71] = 2.0 ** -149
    q = qlr.quantize_i8(x.cuda())
    rq, rs = ref_rows(x)
    assert np.array_equal(q.scale.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(q.q.cpu().numpy().astype(np.float64), rq)


def make(M, N, K, r, seed, xdt="bf16"):
    x, w = rand(M, K, seed, xdt), rand(N, K, seed + 1, "f32", 0.02)
    A = rand(r, K, seed + 2, "bf16", K ** -0.5) if r else None
    B = rand(N, r, seed + 3, "bf16", 0.1) if r else None
    return x, w, A, B


def reference(x, w, A, B, scale):
    """y and its tolerance (before the output's own rounding) in 64 bits."""
    xq, sx = ref_rows(x)
    wq, sw = ref_rows(w)
    y = torch.from_numpy(xq) @ torch.from_numpy(wq).t() * torch.from_numpy(sx.astype(np.float64))[:, None]
    y = y * torch.from_numpy(sw.astype(np.float64))
    tol = 4e-7 * y.abs() + 1e-30
    if A is not None:
        x, A, B = x.double(), A.double(), B.double()
        y = y + scale * (x @ A.t()) @ B.t()
        tol = tol + 1e-4 * abs(scale) * (x.abs() @ A.abs().t()) @ B.abs().t() + 4e-7 * y.abs()
    return y, tol


def check(y, ref, tol):
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs()
    err = (y.double().cpu() - ref).abs()
    assert torch.isfinite(y).all()
    assert (err <= tol).all(), f"worst {(err / tol).max().item():.3g} of the tolerance"


def dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("path,M", [("gemv", 1), ("gemv", 3), ("gemv", 16), ("gemm", 1), ("gemm", 65), ("gemm", 256),
                                    ("auto", 17), ("auto", 300)])
@pytest.mark.parametrize("N,K", [(1, 16), (40, 144), (257, 64), (300, 1040), (513, 4096)])
@pytest.mark.parametrize("r,out", [(0, "f32"), (16, "bf16"), (5, "f32"), (40, "bf16")])
def test_linear(path, M, N, K, r, out):
    print(f"linear_i8 {path} M={M} N={N} K={K} r={r} {out}", flush=True)
    x, w, A, B = make(M, N, K, r, seed=M + N + K + r)
    scale = 0.5
    xd, wd, Ad, Bd = dev(x, w, A, B)
    w8 = qlr.quantize_i8(wd)
    with qlr.path({"gemv": qlr.PATH_GEMV, "gemm": qlr.PATH_GEMM, "auto": qlr.PATH_AUTO}[path]):
        y = qlr.linear_i8(xd, w8, Ad, Bd, scale, out_dtype=DT[out])
    torch.cuda.synchronize()
    check(y, *reference(x, w, A, B, scale))


@pytest.mark.parametrize("M", [2, 130])
def test_given_tokens_and_own_tokens_agree(M):
    x, w, A, B = make(M, 96, 512, 8, seed=4)
    xd, wd, Ad, Bd = dev(x, w, A, B)
    w8, xq = qlr.quantize_i8(wd), qlr.quantize_i8(xd)
    a = qlr.linear_i8(xd, w8, Ad, Bd, 2.0)
    b = qlr.linear_i8(xd, w8, Ad, Bd, 2.0, xq=xq)
    c = qlr.linear_i8(None, w8, xq=xq, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    check(c, *reference(x, w, None, None, 0))


@pytest.mark.parametrize("M", [4, 70])
def test_families_agree_without_adapter(M):
    """Integer sums are exact: the two kernel families give the same bits."""
    x, w, _, _ = make(M, 333, 2064, 0, seed=M)
    xd, wd = dev(x, w)
    w8 = qlr.quantize_i8(wd)
    ys = []
    for m0 in range(0, M, 16):
        with qlr.path(qlr.PATH_GEMV):
            ys.append(qlr.linear_i8(xd[m0:m0 + 16], w8, out_dtype=torch.float32))
    with qlr.path(qlr.PATH_GEMM):
        y = qlr.linear_i8(xd, w8, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(ys), y)


@pytest.mark.parametrize("M,N", [(700, 24576), (2060, 8000), (300, 25000), (520, 33000)])
def test_large_tiles_and_their_rest(M, N):
    """256 x 256 tiles: 3 x 96 = 256 + 32, 9 x 32 = 256 + 32 (odd rows), 2 x 98 = 196 (one round), 3 x 129 = 256 + 131."""
    x, w, A, B = make(M, N, 128, 8, seed=N)
    xd, wd, Ad, Bd = dev(x, w, A, B)
    y = qlr.linear_i8(xd, qlr.quantize_i8(wd), Ad, Bd, 0.5)
    torch.cuda.synchronize()
    check(y, *reference(x, w, A, B, 0.5))


def test_rows_past_32_bit_offsets():
    """Tokens and outputs past 2^32 bytes: the last rows against 64 bits."""
    M, N, K = 540_000, 2064, 8192
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.empty((M, K), dtype=torch.int8, device="cuda")
    q.random_(-127, 128, generator=g)
    s = torch.rand(M, generator=g, device="cuda") + 0.5
    assert q.numel() > 1 << 32
    w = rand(N, K, 7, "f32", 0.02)
    w8 = qlr.quantize_i8(w.cuda())
    y = qlr.linear_i8(None, w8, xq=qlr.I8Rows(M, K, q, s), out_dtype=torch.float32)
    assert y.numel() * 4 > 1 << 32
    torch.cuda.synchronize()
    wq, sw = ref_rows(w)
    for rows in (slice(0, 40), slice(M - 40, M)):
        ref = q[rows].cpu().double() @ torch.from_numpy(wq).t() * s[rows].cpu().double()[:, None]
        ref = ref * torch.from_numpy(sw.astype(np.float64))
        check(y[rows], ref, 4e-7 * ref.abs() + 1e-30)


def test_largest_sums_do_not_wrap():
    """Every product 127 * 127 with one sign over the longest row allowed: 2 114 060 288 < 2^31."""
    K = 131072
    x = torch.ones((18, K), dtype=torch.float32)
    w = torch.ones((24, K), dtype=torch.float32)
    w[1::2] = -1
    xd, wd = dev(x, w)
    w8 = qlr.quantize_i8(wd)
    for m in (3, 18):
        y = qlr.linear_i8(xd[:m], w8, out_dtype=torch.float32)
        torch.cuda.synchronize()
        check(y, *reference(x[:m], w, None, None, 0))


@pytest.mark.parametrize("M", [5, 40])
def test_bad_rows_stay_their_own(M):
    """A token with a NaN gives a NaN row, a zero token a zero row, and a NaN channel a NaN column; the rest is untouched."""
    x, w, _, _ = make(M, 48, 256, 0, seed=9)
    clean = x.clone()
    x[1, 3] = float("nan")
    x[2] = 0
    w[7, 0] = float("inf")
    xd, wd = dev(x, w)
    y = qlr.linear_i8(xd, qlr.quantize_i8(wd), out_dtype=torch.float32).cpu()
    w[7, 0] = 0
    ref, tol = reference(clean, w, None, None, 0)
    assert torch.isnan(y[1]).all() and torch.isnan(y[:, 7]).all()
    ok = torch.ones_like(ref, dtype=torch.bool)
    ok[1] = ok[2] = False
    ok[:, 7] = False
    assert ((y.double() - ref).abs() <= tol)[ok].all()
    keep = torch.arange(48) != 7
    assert (y[2, keep] == 0).all()


def test_float32_tokens_and_no_rows():
    x, w, A, B = make(20, 64, 192, 4, seed=11, xdt="f32")
    xd, wd, Ad, Bd = dev(x, w, A, B)
    w8 = qlr.quantize_i8(wd)
    check(qlr.linear_i8(xd, w8, Ad, Bd, 1.5), *reference(x, w, A, B, 1.5))
    assert qlr.linear_i8(xd[:0], w8, Ad, Bd, 1.5).shape == (0, 64)
    assert qlr.quantize_i8(xd[:0]).q.shape == (0, 192)


def test_captured_call_replays_with_new_tokens():
    x, w, A, B = make(6, 80, 320, 8, seed=21)
    xd, wd, Ad, Bd = dev(x, w, A, B)
    w8 = qlr.quantize_i8(wd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call = qlr.LinearI8Call(xd, w8, Ad, Bd, 0.7)
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    for k in range(4):
        x2 = rand(6, 320, 100 + k)
        xd.copy_(x2.cuda())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = call.y.clone()
        assert torch.equal(got, qlr.linear_i8(xd, w8, Ad, Bd, 0.7))
        check(got, *reference(x2, w, A, B, 0.7))
