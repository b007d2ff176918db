"""The tiled product's waits, counted in the compiled code.

The kernels of qlr_tile.h load x (and 8-bit weights) straight into LDS one to three steps ahead and end each step with a wait
that leaves the newest n vector loads open, then a barrier.  Vector loads return in order, so the wait covers the loads
that the next step reads exactly if at least n vector loads were issued after them.  This test compiles the kernels to
assembly and counts them in every main loop, for every kind, code width and tile.  (No GPU.)"""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from quantized_base_fine_amd import build

KERNEL = re.compile(r"^_ZN3qlr12_GLOBAL__N_16k_tileILi(\d)ELi(\d)ELi(\d+)ELi(\d+)EEE\S*:")


def ahead(kind, bm):
    """Steps between a direct load and its use."""
    return 1 if bm > 64 else 2 if kind == 0 else 3


def direct_loads(kind, bm, bn):
    """Direct loads of a wave in one step."""
    return bm // 64 + (bn // 64 if kind == 0 else 0)


def events(lines):
    """(label, None), ("D"), ("G"), ("W", n), ("B"), ("M"), ("J", label) of a kernel's instructions."""
    out = []
    for line in lines:
        m = re.match(r"^(\.LBB\S+):", line)
        if m:
            out.append(("L", m.group(1)))
            continue
        t = line.split(";")[0].split()
        if not t or not re.match(r"^[a-z]", t[0]):
            continue
        op = t[0]
        if re.match(r"(global|buffer|flat|scratch)_(store|atomic)", op):
            out.append(("S", None))
        elif re.match(r"(global|buffer|flat|scratch)_load", op):
            out.append(("D" if "lds" in t[1:] or "_lds_" in op else "G", None))
        elif op == "s_waitcnt":
            n = re.search(r"vmcnt\((\d+)\)", line)
            if n:
                out.append(("W", int(n.group(1))))
        elif op == "s_barrier":
            out.append(("B", None))
        elif "mfma" in op:
            out.append(("M", None))
        elif op.startswith(("s_cbranch", "s_branch")):
            out.append(("J", t[1]))
    return out


def main_loop(ev):
    """The events of the loop that holds most products."""
    at = {v: i for i, (k, v) in enumerate(ev) if k == "L"}
    best = []
    for i, (k, v) in enumerate(ev):
        if k == "J" and at.get(v, i) < i:
            body = ev[at[v]:i]
            n = sum(x[0] == "M" for x in body)
            if n and (not best or n > sum(x[0] == "M" for x in best)):
                best = body
    return best


def check_loop(body, steps_ahead, per_step):
    """Every barrier of a steady loop: the loads issued after those that the next step reads number at least the wait's count.
    Returns the number of barriers checked."""
    assert sum(k == "D" for k, _ in body) == per_step * sum(k == "B" for k, _ in body), "direct loads of a step"
    assert not any(k == "S" for k, _ in body)  # (stores would count too)
    two, checked = body * 4, 0
    for i in range(3 * len(body), len(two)):
        if two[i][0] != "B":
            continue
        j = i - 1
        while two[j][0] not in "WDG":
            j -= 1
        assert two[j][0] == "W", "a load between the wait and the barrier, or none"
        n, loads, skip = two[j][1], 0, (steps_ahead - 1) * per_step
        while True:
            j -= 1
            if two[j][0] == "D":
                if skip == 0:
                    break
                skip -= 1
            loads += two[j][0] in "DG"
        assert loads >= n, f"wait leaves {n} loads open, only {loads} are newer than those needed"
        checked += 1
    return checked


def assembly(src, out):
    cmd = [build.hipcc(), *build.COMMON, "-S", "--cuda-device-only", os.path.join(build.CSRC, src), "-o", out]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    kernels, name = {}, None
    with open(out) as f:
        for line in f:
            m = KERNEL.match(line)
            if m:
                name = tuple(int(v) for v in m.groups())
                kernels[name] = []
            elif line.startswith(".Lfunc_end"):
                name = None
            elif name is not None:
                kernels[name].append(line)
    return kernels


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    d = tmp_path_factory.mktemp("asm")
    srcs = ["qlr_grouped_fwd.hip", "qlr_grouped_bwd.hip", "qlr_i8.hip"]
    with cf.ThreadPoolExecutor(len(srcs)) as ex:
        parts = list(ex.map(lambda s: assembly(s, str(d / (s + ".s"))), srcs))
    return {k: events(v) for p in parts for k, v in p.items()}


def test_waits_of_every_tile(kernels):
    want = {(k, b, m, n) for k, bits in ((0, [4]), (1, [2, 3, 4, 8]), (2, [2, 3, 4, 8])) for b in bits
            for m, n in ((64, 128), (128, 128), (256, 256))}
    assert set(kernels) == want
    for (kind, bits, bm, bn), ev in sorted(kernels.items()):
        print(kind, bits, bm, bn, flush=True)
        body = main_loop(ev)
        assert check_loop(body, ahead(kind, bm), direct_loads(kind, bm, bn)) >= (2 if bm > 64 else 3)


def test_a_missing_load_is_found(kernels):
    """The count fails with any one code load of a step taken out of a loop that waits by hand, or with a later wait."""
    for key in ((2, 3, 64, 128), (1, 4, 64, 128)):
        body = main_loop(kernels[key])
        g = [i for i, (k, _) in enumerate(body) if k == "G"]
        per = len(g) // sum(k == "B" for k, _ in body)
        assert per >= 3
        if per == 3:
            with pytest.raises(AssertionError):
                check_loop(body[:g[0]] + body[g[0] + 1:], 3, 1)
        late = [("W", v + 8) if k == "W" else (k, v) for k, v in body]
        with pytest.raises(AssertionError):
            check_loop(late, 3, 1)
