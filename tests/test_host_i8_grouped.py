"""Host-side tests of the 8-bit-integer and expert-grouped calls: every refusal (nothing is launched: each call
below fails its checks, or has no rows) and the workspace sizes."""
import ctypes as C

import pytest

from quantized_base_fine_amd import qlr

P = {n: 0x1000000 * (i + 1) for i, n in enumerate(
    ["x", "dy", "w", "s", "A", "B", "y", "dx", "dA", "dB", "ws", "off", "xq", "xs"])}
BF, F16, F32 = qlr.QLR_BF16, qlr.QLR_F16, qlr.QLR_F32


def status(name, *args):
    st = getattr(qlr.lib(), name)(*args)
    return qlr.STATUS[st][4:]


def quant(X=P["x"], dt=F32, rows=4, cols=64, out=(4, 64, P["xq"], P["xs"])):
    o = None if out is None else C.byref(qlr.CI8Rows(*out))
    return status("qlr_quantize_i8", X, dt, rows, cols, o, None)


def test_quantize_refusals():
    assert quant(out=None) == "ERR_NULL" and quant(X=None) == "ERR_NULL"
    assert quant(out=(4, 64, None, P["xs"])) == "ERR_NULL" and quant(out=(4, 64, P["xq"], None)) == "ERR_NULL"
    assert quant(dt=7) == "ERR_DTYPE"
    assert quant(rows=-1) == "ERR_SHAPE" and quant(cols=0) == "ERR_SHAPE" and quant(out=(5, 64, P["xq"], P["xs"])) == "ERR_SHAPE"
    assert quant(X=P["x"] + 8) == "ERR_ALIGN" and quant(out=(4, 64, P["xq"] + 1, P["xs"])) == "ERR_ALIGN"
    assert quant(X=None, rows=0, out=(0, 64, None, None)) == "OK"
    assert quant(out=(4, 64, P["x"], P["xs"])) == "ERR_ALIAS" and quant(out=(4, 64, P["xq"], P["x"] + 1008)) == "ERR_ALIAS"
    assert quant(out=(4, 64, P["xq"], P["xq"] + 240)) == "ERR_ALIAS"


def i8(x=P["x"], xdt=BF, M=4, xq=None, w=(32, 64, P["w"], P["s"]), A=P["A"], B=P["B"], abdt=BF, r=4, y=P["y"], ydt=BF,
       ws=P["ws"], wsb=1 << 30):
    cq = None if xq is None else C.byref(qlr.CI8Rows(*xq))
    cw = None if w is None else C.byref(qlr.CI8Rows(*w))
    return status("qlr_linear_fwd_i8", x, xdt, M, cq, cw, A, B, abdt, r, 1.0, y, ydt, ws, wsb, None)


def test_linear_i8_refusals():
    assert i8(w=None) == "ERR_NULL" and i8(x=None) == "ERR_NULL" and i8(y=None) == "ERR_NULL" and i8(A=None) == "ERR_NULL"
    assert i8(w=(32, 64, None, P["s"])) == "ERR_NULL" and i8(xq=(4, 64, P["xq"], None)) == "ERR_NULL"
    assert i8(x=None, xq=(4, 64, P["xq"], P["xs"])) == "ERR_NULL"  # the adapter needs x
    assert i8(M=-1) == "ERR_SHAPE" and i8(r=-1) == "ERR_SHAPE" and i8(w=(0, 64, P["w"], P["s"])) == "ERR_SHAPE"
    assert i8(w=(32, 72, P["w"], P["s"])) == "ERR_SHAPE" and i8(w=(32, 131088, P["w"], P["s"])) == "ERR_SHAPE"
    assert i8(xq=(5, 64, P["xq"], P["xs"])) == "ERR_SHAPE" and i8(xq=(4, 80, P["xq"], P["xs"])) == "ERR_SHAPE"
    assert i8(xdt=F16) == "ERR_DTYPE" and i8(ydt=F16) == "ERR_DTYPE" and i8(abdt=F32) == "ERR_DTYPE"
    for n in ("x", "A", "B", "y", "ws"):
        assert i8(**{n: P[n] + 4}) == "ERR_ALIGN", n
    need = qlr.workspace_bytes(qlr.OP_LINEAR_I8, 4, 32, 64, 4)
    assert need == 256 + 256 + 256  # t partials (one split at K = 64), int8 tokens, scales, each rounded up
    assert i8(wsb=need - 1) == "ERR_WORKSPACE" and i8(ws=None) == "ERR_WORKSPACE"
    with qlr.path(qlr.PATH_F32):
        assert i8() == "ERR_PATH"
    with qlr.path(qlr.PATH_GEMV):
        assert i8(M=17) == "ERR_PATH"
    assert i8(M=0, x=None, y=None) == "OK"
    assert i8(M=(1 << 27) + 1) == "ERR_SHAPE" and i8(r=(1 << 20) + 1) == "ERR_SHAPE"
    for n in ("x", "w", "s", "A", "B"):
        assert i8(y=P[n]) == "ERR_ALIAS", n
    for n in ("xq", "xs"):
        assert i8(xq=(4, 64, P["xq"], P["xs"]), y=P[n]) == "ERR_ALIAS", n


def grouped(x=P["x"], xdt=BF, T=4, w=None, E=2, off=P["off"], A=P["A"], B=P["B"], abdt=BF, r=4, y=P["y"], ydt=BF,
            ws=P["ws"], wsb=1 << 30, rows=32, cols=64, bits=4, fmt=1):
    cw = qlr.CQWeight(fmt, bits, 64, 256, rows, cols, P["w"], P["s"], P["xs"]) if w is None else w
    return status("qlr_linear_fwd_grouped", x, xdt, T, C.byref(cw), E, off, A, B, abdt, r, 1.0, y, ydt, ws, wsb, None)


def bwd(dy=P["dy"], dydt=BF, x=P["x"], xdt=BF, T=4, E=2, off=P["off"], A=P["A"], B=P["B"], abdt=BF, r=4, dx=P["dx"], dxdt=BF,
        dA=P["dA"], dB=P["dB"], ws=P["ws"], wsb=1 << 30, rows=32, cols=64, bits=4, fmt=1):
    cw = qlr.CQWeight(fmt, bits, 64, 256, rows, cols, P["w"], P["s"], P["xs"])
    return status("qlr_linear_bwd_grouped", dy, dydt, x, xdt, T, C.byref(cw), E, off, A, B, abdt, r, 1.0, dx, dxdt, dA, dB,
                  ws, wsb, None)


@pytest.mark.parametrize("call", [grouped, bwd], ids=["forward", "backward"])
def test_grouped_refusals(call):
    assert call(off=None) == "ERR_NULL" and call(x=None) == "ERR_NULL" and call(A=None) == "ERR_NULL"
    assert call(B=None) == "ERR_NULL"
    assert call(T=-1) == "ERR_SHAPE" and call(T=(1 << 30) + 1) == "ERR_SHAPE" and call(r=-1) == "ERR_SHAPE"
    assert call(E=0) == "ERR_SHAPE" and call(E=3) == "ERR_SHAPE" and call(E=4097, rows=4097 * 8) == "ERR_SHAPE"
    assert call(cols=96) == "ERR_SHAPE" and call(rows=0) == "ERR_SHAPE"
    assert call(xdt=F32) == "ERR_DTYPE" and call(abdt=F32) == "ERR_DTYPE"
    assert call(bits=5) == "ERR_BITS" and call(fmt=2) == "ERR_FORMAT"
    assert call(x=P["x"] + 2) == "ERR_ALIGN" and call(off=P["off"] + 2) == "ERR_ALIGN" and call(B=P["B"] + 2) == "ERR_ALIGN"
    assert call(ws=P["ws"] + 8) == "ERR_ALIGN" and call(wsb=64) == "ERR_WORKSPACE" and call(ws=None) == "ERR_WORKSPACE"
    for p in (qlr.PATH_F32, qlr.PATH_GEMV):
        with qlr.path(p):
            assert call() == "ERR_PATH"


def test_forward_only_refusals():
    assert grouped(y=None) == "ERR_NULL" and grouped(ydt=F16) == "ERR_DTYPE" and grouped(y=P["y"] + 2) == "ERR_ALIGN"
    for n in ("x", "A", "B", "off", "w", "s", "xs"):  # (w, s, xs: the weight's codes, absmax codes and constants)
        assert grouped(y=P[n]) == "ERR_ALIAS", n
    assert grouped(T=(1 << 27) + 1) == "ERR_SHAPE"
    assert grouped(T=0, x=None, y=None) == "OK"


def test_backward_only_refusals():
    assert bwd(dy=None) == "ERR_NULL" and bwd(dA=None) == "ERR_NULL" and bwd(dB=None) == "ERR_NULL"
    assert bwd(rows=2 * 12) == "ERR_SHAPE"  # 12 rows of an expert
    assert bwd(dydt=F32) == "ERR_DTYPE" and bwd(dxdt=F16) == "ERR_DTYPE"
    assert bwd(dx=P["dx"] + 2) == "ERR_ALIGN" and bwd(dA=P["dA"] + 4) == "ERR_ALIGN"
    for o, i in (("dx", "dy"), ("dx", "x"), ("dA", "A"), ("dB", "B"), ("dB", "off"), ("dA", "x"), ("dx", "w"), ("dA", "s"),
                 ("dB", "xs")):
        assert bwd(**{o: P[i]}) == "ERR_ALIAS", (o, i)
    assert bwd(dA=P["dB"]) == "ERR_ALIAS" and bwd(dx=P["dA"]) == "ERR_ALIAS"


def test_grouped_workspace():
    f, b = qlr.OP_LINEAR_GROUPED, qlr.OP_LINEAR_GROUPED_BWD
    ws = qlr.grouped_workspace_bytes
    assert ws(f, 0, 64, 64, 2, 8) == 0 and ws(f, 9, 64, 64, 2, 0) == 0 and ws(b, 9, 64, 64, 2, 0) == 0
    assert ws(f, 100, 64, 64, 2, 8) == 3328                      # 100 x 8 float32, rounded up to 256
    assert ws(b, 100, 64, 64, 2, 8) == 2 * 3328 + 1024           # t, u, B transposed (64 x 8 bf16), no partials
    assert ws(b, 1024, 64, 64, 2, 8) == 2 * 32768 + 1024 + 2 * 8 * (32 + 64) * 4  # two extra 512-row chunks at most
    for args in ((qlr.OP_LINEAR, 1, 64, 64, 2, 8), (f, -1, 64, 64, 2, 8), (f, 1, 64, 64, 0, 8), (f, 1, 65, 64, 2, 8)):
        with pytest.raises(qlr.QlrError):
            ws(*args)


def test_binding_refusals():
    """The binding's own checks: host tensors, types, shapes, packing."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w8 = qlr.I8Rows(32, 64, torch.zeros(32, 64, dtype=torch.int8), torch.zeros(32))
    with pytest.raises(ValueError):
        qlr.quantize_i8(x)  # host memory
    with pytest.raises(ValueError):
        qlr.linear_i8(x, w8)
    with pytest.raises(ValueError):
        qlr.LinearI8Call(None, w8)
    qw = qlr.QWeight(4, 64, 64, *[torch.zeros(1)] * 3)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        qlr.linear_grouped(x, qw, off)
    for bad in (off.long(), off[:1], torch.zeros(2, 3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)):
        with pytest.raises(ValueError):
            qlr._grouped_operands(qw, bad, None, None)
    A, B = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 32, 4, dtype=torch.bfloat16)
    assert qlr._grouped_operands(qw, off, A, B) == (2, 32, 4)
    for a, b in ((A, None), (A[:, :, :32], B), (A.float(), B.float()), (A, B.transpose(1, 2).contiguous()),
                 (A.transpose(0, 1).contiguous().transpose(0, 1), B)):
        with pytest.raises(ValueError):
            qlr._grouped_operands(qw, off, a, b)
    with pytest.raises(ValueError):
        qlr._rows2d(x.t(), "x")
