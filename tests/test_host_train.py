"""Host-side tests of the calls under adapter dropout and of the gated block: every refusal (nothing is launched: each call
below fails its checks, or has no rows) and the workspace sizes."""
import ctypes as C

import pytest

from quantized_base_fine_amd import qlr

P = {n: 0x1000000 * (i + 1) for i, n in enumerate(
    ["x", "dy", "w", "q8", "cst", "A", "B", "y", "gu", "dx", "dA", "dB", "ws", "step"])}
BF, F16, F32 = qlr.QLR_BF16, qlr.QLR_F16, qlr.QLR_F32


def status(name, *args):
    return qlr.STATUS[getattr(qlr.lib(), name)(*args)][4:]


def weight(rows, cols, bits, fmt, w, q8, cst):
    return C.byref(qlr.CQWeight(fmt, bits, 64, 256, rows, cols, w, q8, cst))


def dropout(p, step):
    return None if p is None else C.byref(qlr.CDropout(p, 1, 2, step))


def fwd(x=P["x"], xdt=BF, M=40, A=P["A"], B=P["B"], abdt=BF, r=4, p=0.1, step=None, y=P["y"], ydt=BF, ws=P["ws"], wsb=1 << 40,
        rows=32, cols=64, bits=4, fmt=1, w=P["w"], q8=P["q8"], cst=P["cst"]):
    return status("qlr_linear_fwd_dropout", x, xdt, M, weight(rows, cols, bits, fmt, w, q8, cst), A, B, abdt, r, 1.0,
                  dropout(p, step), y, ydt, ws, wsb, None)


def bwd(dy=P["dy"], dydt=BF, x=P["x"], xdt=BF, M=40, A=P["A"], B=P["B"], abdt=BF, r=4, p=0.1, step=None, dx=P["dx"], dxdt=BF,
        dA=P["dA"], dB=P["dB"], ws=P["ws"], wsb=1 << 40, rows=32, cols=64, bits=4, fmt=1, w=P["w"], q8=P["q8"], cst=P["cst"]):
    return status("qlr_linear_bwd_dropout", dy, dydt, x, xdt, M, weight(rows, cols, bits, fmt, w, q8, cst), A, B, abdt, r, 1.0,
                  dropout(p, step), dx, dxdt, dA, dB, ws, wsb, None)


def gated(x=P["x"], xdt=BF, M=40, act=0, A=P["A"], B=P["B"], abdt=BF, r=4, p=0.1, step=None, y=P["y"], ydt=BF, gu=P["gu"],
          ws=P["ws"], wsb=1 << 40, rows=32, cols=64, bits=4, fmt=1, w=P["w"], q8=P["q8"], cst=P["cst"]):
    return status("qlr_gated_fwd", x, xdt, M, weight(rows, cols, bits, fmt, w, q8, cst), act, A, B, abdt, r, 1.0,
                  dropout(p, step), y, ydt, gu, ws, wsb, None)


def gbwd(dy=P["dy"], dydt=BF, gu=P["gu"], x=P["x"], xdt=BF, M=40, act=0, A=P["A"], B=P["B"], abdt=BF, r=4, p=0.1, step=None,
         dx=P["dx"], dxdt=BF, dA=P["dA"], dB=P["dB"], ws=P["ws"], wsb=1 << 40, rows=32, cols=64, bits=4, fmt=1, w=P["w"],
         q8=P["q8"], cst=P["cst"]):
    return status("qlr_gated_bwd", dy, dydt, gu, x, xdt, M, weight(rows, cols, bits, fmt, w, q8, cst), act, A, B, abdt, r, 1.0,
                  dropout(p, step), dx, dxdt, dA, dB, ws, wsb, None)


CALLS = pytest.mark.parametrize("call", [fwd, bwd, gated, gbwd], ids=["layer", "layer bwd", "block", "block bwd"])
BACKWARD = pytest.mark.parametrize("call", [bwd, gbwd], ids=["layer", "block"])


@CALLS
def test_refusals_of_all(call):
    assert call(x=None) == "ERR_NULL" and call(A=None) == "ERR_NULL" and call(B=None) == "ERR_NULL" and call(w=None) == "ERR_NULL"
    assert call(M=-1) == "ERR_SHAPE" and call(M=(1 << 27) + 1) == "ERR_SHAPE"
    assert call(r=-1) == "ERR_SHAPE" and call(r=(1 << 20) + 1) == "ERR_SHAPE"
    assert call(cols=96) == "ERR_SHAPE" and call(rows=0) == "ERR_SHAPE" and call(cols=0) == "ERR_SHAPE"
    assert call(rows=(1 << 20) + 16) == "ERR_SHAPE" and call(cols=(1 << 20) + 64) == "ERR_SHAPE"
    assert call(M=1 << 27, cols=1 << 19) == "ERR_SHAPE"  # (2^46 elements of x)
    assert call(xdt=F32) == "ERR_DTYPE" and call(abdt=F32) == "ERR_DTYPE" and call(abdt=F16) == "ERR_DTYPE"
    assert call(bits=5) == "ERR_BITS" and call(fmt=2) == "ERR_FORMAT"
    for n in ("x", "A", "B", "w", "q8", "cst", "ws"):
        assert call(**{n: P[n] + 8}) == "ERR_ALIGN", n
    assert call(wsb=64) == "ERR_WORKSPACE" and call(ws=None) == "ERR_WORKSPACE"
    with qlr.path(qlr.PATH_F32):
        assert call is fwd or call() == "ERR_PATH"
    with qlr.path(qlr.PATH_GEMV):
        assert call() == "ERR_PATH"  # (40 rows)


@CALLS
@pytest.mark.parametrize("p", [-1e-9, 1.0, 1.5, float("nan"), float("inf")])
def test_dropout_refusals(call, p):
    assert call(p=p) == "ERR_VALUE" and call(p=p, r=0, A=None, B=None) == "ERR_VALUE"


@CALLS
def test_step_refusals(call):
    assert call(step=P["step"] + 4) == "ERR_ALIGN"
    out = "dx" if call in (bwd, gbwd) else "y"
    assert call(step=P[out] + 8) == "ERR_ALIAS"  # an output over the step


def test_forward_refusals():
    for call in (fwd, gated):
        assert call(y=None) == "ERR_NULL" and call(y=P["y"] + 2) == "ERR_ALIGN" and call(ydt=F16) == "ERR_DTYPE"
        for n in ("x", "w", "q8", "cst", "A", "B", "ws"):
            assert call(y=P[n]) == "ERR_ALIAS", n
        assert call(M=0, x=None, y=None) == "OK"


@pytest.mark.parametrize("call", [gated, gbwd], ids=["forward", "backward"])
def test_block_refusals(call):
    assert call(rows=33) == "ERR_SHAPE"
    assert call(act=-1) == "ERR_VALUE" and call(act=3) == "ERR_VALUE"
    assert call(gu=P["gu"] + 2) == "ERR_ALIGN"


def test_block_outputs():
    for n in ("x", "w", "q8", "cst", "A", "B", "ws", "y"):
        assert gated(gu=P[n]) == "ERR_ALIAS", n
    assert gbwd(gu=None) == "ERR_NULL"
    assert gated(M=0, x=None, y=None, gu=None) == "OK"


@BACKWARD
def test_backward_refusals(call):
    assert call(dy=None) == "ERR_NULL" and call(dA=None) == "ERR_NULL" and call(dB=None) == "ERR_NULL"
    assert call(rows=12 if call is bwd else 24) == "ERR_SHAPE"  # 12 columns of dy
    assert call(dydt=F32) == "ERR_DTYPE" and call(dxdt=F16) == "ERR_DTYPE"
    assert call(dy=P["dy"] + 2) == "ERR_ALIGN" and call(dx=P["dx"] + 2) == "ERR_ALIGN" and call(dA=P["dA"] + 4) == "ERR_ALIGN"
    inputs = ["dy", "x", "w", "q8", "cst", "A", "B", "ws"] + (["gu"] if call is gbwd else [])
    for o in ("dx", "dA", "dB"):
        for i in inputs:
            assert call(**{o: P[i]}) == "ERR_ALIAS", (o, i)
    assert call(dA=P["dB"]) == "ERR_ALIAS" and call(dx=P["dA"]) == "ERR_ALIAS" and call(dx=P["dB"]) == "ERR_ALIAS"


def test_workspace():
    ws = qlr.workspace_bytes
    d, db, g, gb = qlr.OP_LINEAR_DROPOUT, qlr.OP_LINEAR_DROPOUT_BWD, qlr.OP_GATED, qlr.OP_GATED_BWD
    for op in (d, db, g, gb):
        assert ws(op, 0, 64, 64, 8) == 0
        for args in ((-1, 64, 64, 8), (4, -8, 64, 8), (4, 64, 64, -1)):
            with pytest.raises(qlr.QlrError):
                ws(op, *args)
    for op in (d, db, g):
        assert ws(op, 9, 64, 64, 0) == 0
    assert ws(gb, 9, 64, 64, 0) == 9 * 128 * 2               # dgu, bf16 (256-byte pieces)
    assert ws(d, 100, 64, 64, 8) == 3328                      # t: 100 x 8 float32, rounded up to 256
    assert ws(db, 100, 64, 64, 8) == 2 * 3328 + 1024 + 4096   # t, u, the mask's bits (100 x 8), one chunk more of dA and dB
    # a dense bf16 copy of the weight from 1536 rows on where the products are large
    big, small = ws(g, 1536, 11008, 4096, 0), ws(g, 1535, 11008, 4096, 0)
    assert small == 0 and big >= 2 * 11008 * 4096 * 2


def test_binding_refusals():
    """The binding's own checks: host tensors, types, shapes, packing."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    qw = qlr.QWeight(4, 32, 64, *[torch.zeros(1)] * 3)
    for call in (qlr.linear_dropout, qlr.gated):
        with pytest.raises(ValueError):
            call(x, qw)  # host memory
    with pytest.raises(ValueError):
        qlr.linear_dropout_bwd(x[:, :32].contiguous(), x, qw)
    with pytest.raises(ValueError):
        qlr.gated_bwd(x[:, :16].contiguous(), x[:, :32].contiguous(), x, qw)
    with pytest.raises(ValueError):
        qlr.Dropout(0.1, 1, 0, torch.zeros(1, dtype=torch.int64)).c_struct()  # the step in host memory
    assert "ERR_VALUE" in qlr.STATUS[13] and set(qlr.ACTIVATIONS) == {"silu", "gelu", "gelu_tanh"}
