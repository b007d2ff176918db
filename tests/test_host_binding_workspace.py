"""Host-side test: a workspace tensor whose elements do not lie one after another (an expanded one has fewer bytes behind it than
elements) is refused by every call that takes one, before anything is launched."""
import pytest

torch = pytest.importorskip("torch")

from quantized_base_fine_amd import qlr  # noqa: E402

BF = torch.bfloat16
WIDE = torch.zeros(1, dtype=torch.uint8).expand(1 << 30)


def weight(rows=32, cols=64):
    return qlr.QWeight(4, rows, cols, torch.zeros(rows * cols // 2, dtype=torch.uint8), torch.zeros(rows, dtype=torch.uint8),
                       torch.zeros(1))


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


SP = lambda: qlr.Sparse(32, 64, 1, torch.zeros(33, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1))  # noqa: E731
OFF = lambda: torch.tensor([0, 4], dtype=torch.int32)  # noqa: E731
I8 = lambda: qlr.I8Rows(32, 64, torch.zeros((32, 64), dtype=torch.int8), torch.zeros(32))  # noqa: E731
CALLS = {
    "quantize": lambda ws: qlr.quantize(z(32, 64), 4, ws=ws),
    "linear": lambda ws: qlr.linear(z(4, 64), weight(), z(8, 64), z(32, 8), 1.0, ws=ws),
    "linear call": lambda ws: qlr.LinearCall(z(4, 64), weight(), z(8, 64), z(32, 8), 1.0, ws=ws),
    "mixed": lambda ws: qlr.MixedCall([dict(x=z(4, 64), qw=weight(), A=z(8, 64), B=z(32, 8), scale=1.0)], ws=ws),
    "linear bwd": lambda ws: qlr.LinearBwdCall(z(4, 32), z(4, 64), weight(), z(8, 64), z(32, 8), 1.0, ws=ws),
    "outliers": lambda ws: qlr.quantize_outliers(z(32, 64), 4, 1, ws=ws),
    "linear outliers": lambda ws: qlr.OutliersCall(z(4, 64), weight(), SP(), z(8, 64), z(32, 8), 1.0, ws=ws),
    "wha": lambda ws: qlr.WhaCall(z(4, 64), weight(), SP(), 64, ws=ws),
    "i8": lambda ws: qlr.LinearI8Call(z(4, 64), I8(), ws=ws),
    "grouped": lambda ws: qlr.GroupedCall(z(4, 64), weight(), OFF(), z(1, 8, 64), z(1, 32, 8), 1.0, ws=ws),
    "grouped bwd": lambda ws: qlr.GroupedBwdCall(z(4, 32), z(4, 64), weight(), OFF(), z(1, 8, 64), z(1, 32, 8), 1.0, ws=ws),
    "dropout": lambda ws: qlr.LinearDropoutCall(z(4, 64), weight(), z(8, 64), z(32, 8), 1.0, ws=ws),
    "dropout bwd": lambda ws: qlr.LinearDropoutBwdCall(z(4, 32), z(4, 64), weight(), z(8, 64), z(32, 8), 1.0, ws=ws),
    "gated": lambda ws: qlr.GatedCall(z(4, 64), weight(), z(2, 8, 64), z(2, 16, 8), 1.0, ws=ws),
    "gated bwd": lambda ws: qlr.GatedBwdCall(z(4, 16), z(4, 32), z(4, 64), weight(), z(2, 8, 64), z(2, 16, 8), 1.0, ws=ws),
}


@pytest.mark.parametrize("name", CALLS)
def test_workspace_of_fewer_bytes_than_elements(monkeypatch, name):
    class Launched(Exception):
        pass

    def reached(*a):
        raise Launched

    monkeypatch.setattr(qlr, "_require_cuda", lambda *t: None)
    monkeypatch.setattr(qlr, "_stream", reached)  # the last thing that a call looks up before its launch
    with pytest.raises(Launched):
        CALLS[name](torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="ws must be contiguous"):
        CALLS[name](WIDE)
