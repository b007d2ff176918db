"""GPU test: the few-rows calls from several host threads at once, each on its own stream with its own workspace and outputs, give
what one thread gives."""
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from quantized_base_fine_amd import qlr  # noqa: E402
from train_ref import Train  # noqa: E402


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
def test_decode_from_four_threads(bits):
    layers = [Train(M, 104, 512, bits, 8, seed=M, sides=2) for M in (1, 4, 9, 16)]
    want = [qlr.gated(L.xd, L.qw, L.Ad, L.Bd, L.scale) for L in layers]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def run(i):
        try:
            L, s = layers[i], torch.cuda.Stream()
            with torch.cuda.stream(s):
                call = qlr.GatedCall(L.xd, L.qw, L.Ad, L.Bd, L.scale)
                for _ in range(20):
                    got[i] = call()
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert all(torch.equal(a, b) for a, b in zip(got, want))
