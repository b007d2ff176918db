"""The waits of the dense product and of the tiled product's newer kinds, counted in the compiled code.

Both load straight into LDS ahead of their use and end each part of a step with a wait that leaves the newest n vector loads
open.  Vector loads return in order, so a wait covers the loads that are read behind it exactly if at least n were issued
after them.  (No GPU.)"""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

import test_host_tile_waits as tiles
from quantized_base_fine_amd import build

KINDS = {3: "qlr_gated_fwd.hip", 4: "qlr_drop_dx.hip", 5: "qlr_drop_fwd.hip"}


def dense_assembly(src, out):
    cmd = [build.hipcc(), *build.COMMON, "-S", "--cuda-device-only", os.path.join(build.CSRC, src), "-o", out]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    kernels, name = {}, None
    with open(out) as f:
        for line in f:
            m = re.match(r"^_ZN3qlr12_GLOBAL__N_17k_denseILi(\d)EEE\S*:", line)
            if m:
                name = int(m.group(1))
                kernels[name] = []
            elif line.startswith(".Lfunc_end"):
                name = None
            elif name is not None:
                kernels[name].append(line)
    return kernels


def steady_loop(ev, products):
    """The shortest loop of so many products with a barrier in it (jumps back to code laid out before it span more)."""
    at = {v: i for i, (k, v) in enumerate(ev) if k == "L"}
    bodies = [ev[at[v]:i] for i, (k, v) in enumerate(ev) if k == "J" and at.get(v, i) < i]
    bodies = [b for b in bodies if sum(k == "M" for k, _ in b) == products and any(k == "B" for k, _ in b)]
    assert bodies, products
    return min(bodies, key=len)


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    d = tmp_path_factory.mktemp("asm")
    with cf.ThreadPoolExecutor(4) as ex:
        jobs = [ex.submit(tiles.assembly, s, str(d / (s + ".s"))) for s in KINDS.values()]
        dense = ex.submit(dense_assembly, "qlr_dense.hip", str(d / "dense.s"))
        parts = [j.result() for j in jobs]
        return {k: tiles.events(v) for p in parts for k, v in p.items()}, {k: tiles.events(v) for k, v in dense.result().items()}


def test_waits_of_the_tiles(compiled):
    kernels = compiled[0]
    assert set(kernels) == {(k, b, m, n) for k in KINDS for b in (2, 3, 4, 8) for m, n in ((64, 128), (128, 128), (256, 256))
                            if (k, m) != (5, 256)}
    for (kind, bits, bm, bn), ev in sorted(kernels.items()):
        print(kind, bits, bm, bn, flush=True)
        # 32 x 32 x 16 products of a wave in the loop's steps, four for the 64-row tiles, else two
        body = steady_loop(ev, (bm * bn * 64) // (8 * 32 * 32 * 16) * (4 if bm == 64 else 2))
        assert tiles.check_loop(body, tiles.ahead(kind, bm), tiles.direct_loads(kind, bm, bn)) >= (2 if bm > 64 else 3)


def test_waits_of_the_dense_product(compiled):
    """Two steps of two halves each: in every half 4 direct loads (two pieces of two) and a wait that leaves 8 open; the pieces
    that a half reads were loaded three halves before its barrier."""
    kernels = compiled[1]
    assert set(kernels) == {0, 1, 2}
    for kind, ev in sorted(kernels.items()):
        body = steady_loop(ev, 128)
        ops = [k for k, _ in body]
        assert ops.count("B") == 4 and ops.count("M") == 128 and "S" not in ops and "G" not in ops, kind
        halves, loads, wait = [], 0, None
        for k, n in body:
            if k == "D":
                loads += 1
            elif k == "W":
                wait = n
            elif k == "B":
                halves.append((loads, wait))
                loads, wait = 0, None
        assert loads == 0 and halves == [(4, 8)] * 4, (kind, halves)
