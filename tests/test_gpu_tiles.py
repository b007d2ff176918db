"""GPU tests of tile shapes and borders that the other tests of the 8-bit-integer and expert-grouped calls do not reach:
128 x 128 tiles as a whole call, malformed offsets over long ranges, the largest integer sums with -128, the most experts, wide
adapters and the longest rows.  Oracles and tolerances of test_gpu_grouped.py and test_gpu_i8.py."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from test_gpu_grouped import BF, F32, Layer, check_backward, check_forward  # noqa: E402
from test_gpu_i8 import check, make, reference  # noqa: E402


@pytest.mark.parametrize("m,K,wv,xv", [(3, 131056, -128, -128), (18, 131056, -128, -128), (3, 131072, -128, 127),
                                       (18, 131072, -128, 127), (18, 131072, 127, -128)])
def test_largest_sums_with_minus_128(m, K, wv, xv):
    """128 * 128 * 131056 = 2 147 221 504 < 2^31, the largest K (a multiple of 16) for -128 in both operands."""
    print(f"linear_i8 M={m} K={K} w={wv} x={xv}", flush=True)
    w8, xq = qlr.I8Rows.empty(24, K, "cuda"), qlr.I8Rows.empty(m, K, "cuda")
    w8.q.fill_(wv), xq.q.fill_(xv), w8.scale.fill_(0.5), xq.scale.fill_(0.25)
    y = qlr.linear_i8(None, w8, xq=xq, out_dtype=F32)
    torch.cuda.synchronize()
    ref = torch.full((m, 24), float(wv * xv * K) * 0.125, dtype=torch.float64)
    check(y, ref, 4e-7 * ref.abs())


@pytest.mark.parametrize("M,N,K,r,out", [(2047, 4096, 128, 8, BF), (2047, 4096, 400, 5, F32), (1024, 4090, 272, 0, F32)])
def test_i8_on_128_x_128_tiles(M, N, K, r, out):
    """16 or 8 row tiles x 32 column tiles of 128 (at most 128 tiles of 256 x 256, too few)."""
    print(f"linear_i8 M={M} N={N} K={K} r={r}", flush=True)
    x, w, A, B = make(M, N, K, r, seed=M + K)
    up = [None if t is None else t.cuda() for t in (x, w, A, B)]
    y = qlr.linear_i8(up[0], qlr.quantize_i8(up[1]), up[2], up[3], 0.5, out_dtype=out)
    torch.cuda.synchronize()
    check(y, *reference(x, w, A, B, 0.5))


@pytest.mark.parametrize("r", [8, 35])
@pytest.mark.parametrize("bits", [2, 3, 4, 8])
def test_grouped_on_128_x_128_tiles(bits, r):
    """600 rows in 4 ranges on 64 column tiles of 128: estimated at 384 tiles (0.59 rounds) against 128 of 256 x 256 (1 round);
    ranges of two tiles, the second of 3 to 72 rows."""
    print(f"grouped on 128 x 128 tiles, bits={bits} r={r}", flush=True)
    counts = [150, 131, 200, 119]
    check_forward(Layer(counts, 8192, 320, bits, r, seed=bits + r, lead=1, pad=2))
    check_backward(Layer(counts, 200, 8192, bits, r, seed=bits + r, lead=1, pad=2))


@pytest.mark.parametrize("r", [8, 12])
@pytest.mark.parametrize("bad", [[0, 1500, 0, 1500], [700, 1500, 100, 1400], [1500, 0, 1500, 0], [-3, 1600, -9, 1 << 30],
                                 [0, 1024, 500, 2000]], ids=str)
def test_malformed_offsets_over_long_ranges(bad, r):
    """Overlapping ranges of more than one gradient chunk (512 rows), so more chunks than the workspace holds: nothing outside
    y, dx, dA, dB and the workspace is written."""
    print(f"grouped offsets={bad} r={r}", flush=True)
    L = Layer([500, 600, 400], 48, 128, 4, r, seed=2)
    L.offsets.copy_(torch.tensor(bad, dtype=torch.int32))
    guard = 4096  # bytes on either side

    def guarded(shape, dtype):
        n = 1
        for s in shape:
            n *= s
        size = torch.empty(0, dtype=dtype).element_size() * n
        buf = torch.full((guard + (size + 255) // 256 * 256 + guard,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, size, buf[guard:guard + size].view(dtype).view(shape)

    need = [qlr.grouped_workspace_bytes(op, L.T, L.E * L.N, L.K, L.E, r) for op in (qlr.OP_LINEAR_GROUPED, qlr.OP_LINEAR_GROUPED_BWD)]
    bufs = [guarded(s, d) for s, d in (((L.T, L.N), BF), ((L.T, L.K), BF), ((L.E, r, L.K), F32), ((L.E, L.N, r), F32),
                                       ((need[0],), torch.uint8), ((need[1],), torch.uint8))]
    y, dx, dA, dB, w0, w1 = (b[2] for b in bufs)
    qlr.GroupedCall(L.xd, L.qw, L.offsets, L.Ad, L.Bd, 1.0, out=y, ws=w0)()
    qlr.GroupedBwdCall(L.dyd, L.xd, L.qw, L.offsets, L.Ad, L.Bd, 1.0, dx=dx, dA=dA, dB=dB, ws=w1)()
    torch.cuda.synchronize()
    for buf, size, _ in bufs:
        assert (buf[:guard] == 0xA5).all() and (buf[guard + size:] == 0xA5).all()


@pytest.mark.parametrize("path", ["auto", "gemm"])
def test_the_most_experts(path):
    """4096 experts: most without rows, some of 1 to 5, one of 17 and one of 700 (two gradient chunks)."""
    counts = [(i * i) % 7 % 6 if i % 9 == 0 else 0 for i in range(qlr.MAX_EXPERTS)]
    counts[1000], counts[4095] = 17, 700
    print(f"grouped, {len(counts)} experts, {sum(counts)} rows, {path}", flush=True)
    L = Layer(counts, 8, 64, 4, 4, seed=17, pad=2)
    check_forward(L, path)
    check_backward(L)


@pytest.mark.parametrize("r", [136, 257])
def test_wide_ranks(r):
    """More than two blocks of 64 adapter columns, and a rank that is no multiple of 8."""
    print(f"grouped r={r}", flush=True)
    L = Layer([9, 0, 16, 200, 530], 72, 192, 4, r, seed=r, pad=1)
    check_forward(L)
    check_backward(L)


@pytest.mark.parametrize("K,N", [(1 << 20, 16), (64, 1 << 20)])
def test_longest_rows(K, N):
    """The longest rows of x and of dy (2^21 bytes): the few-rows kernel, the tiles and the gradients."""
    print(f"grouped N={N} K={K}", flush=True)
    L = Layer([12, 30], N, K, 4, 8, seed=23)
    check_forward(L)
    check_backward(L)
