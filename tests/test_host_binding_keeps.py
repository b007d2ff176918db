"""Host-side test: a prepared call keeps the tensors whose addresses it holds, also when the fields of the weight, the sparse
entries, the 8-bit rows or the dropout that it was made from are set to other tensors afterwards (nothing is launched)."""
import gc
import weakref

import pytest

torch = pytest.importorskip("torch")

from quantized_base_fine_amd import qlr  # noqa: E402


@pytest.fixture
def host(monkeypatch):
    """The binding's checks pass for host tensors."""
    monkeypatch.setattr(qlr, "_require_cuda", lambda *t: None)


def weight():
    return qlr.QWeight(4, 32, 64, torch.zeros(1024, dtype=torch.uint8), torch.zeros(32, dtype=torch.uint8), torch.zeros(1))


CASES = {
    "weight": (weight, ["codes", "absmax_q8", "absmax_c"]),
    "sparse": (lambda: qlr.Sparse(2, 8, 1, torch.zeros(3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1)),
               ["row_ptr", "col", "val"]),
    "i8": (lambda: qlr.I8Rows(2, 16, torch.zeros((2, 16), dtype=torch.int8), torch.zeros(2)), ["q", "scale"]),
    "dropout": (lambda: qlr.Dropout(0.1, 1, 2, torch.zeros(1, dtype=torch.int64)), ["step"]),
}


@pytest.mark.parametrize("name", CASES)
def test_structures_keep_their_tensors(host, name):
    make, fields = CASES[name]
    o = make()
    refs = [weakref.ref(getattr(o, f)) for f in fields]
    c = o.c_struct()
    for f in fields:
        setattr(o, f, None)
    gc.collect()
    assert all(r() is not None for r in refs)
    del c
    gc.collect()
    assert all(r() is None for r in refs)


def test_calls_under_dropout_keep_the_step(host, monkeypatch):
    monkeypatch.setattr(qlr, "_stream", lambda *d: None)
    monkeypatch.setattr(qlr, "_Launch", lambda fn, args, device: None)
    x, h = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((4, 32), dtype=torch.bfloat16)
    for make in (lambda d: qlr.LinearDropoutCall(x, weight(), dropout=d), lambda d: qlr.LinearDropoutBwdCall(h, x, weight(), dropout=d),
                 lambda d: qlr.GatedCall(x, weight(), dropout=d),
                 lambda d: qlr.GatedBwdCall(h[:, :16].contiguous(), h, x, weight(), dropout=d)):
        d = qlr.Dropout(0.1, 1, 2, torch.zeros(1, dtype=torch.int64))
        step = weakref.ref(d.step)
        call = make(d)
        d.step = None  # a next step's, say
        gc.collect()
        assert step() is not None
        del call
        gc.collect()
        assert step() is None
