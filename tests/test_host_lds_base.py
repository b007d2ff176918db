"""Kernels that read LDS at addresses of their own (a level table from byte 0) have no static LDS, which would lie there.

In the compiler's intermediate code such an address is an integer converted to a pointer of address space 3; the static LDS
of a kernel stands in its descriptor.  The launchers check it at run time; this test finds it when the kernels
are built.  (No GPU.)"""
import concurrent.futures as cf
import os
import re
import subprocess

from quantized_base_fine_amd import build

SOURCES = ["qlr_grouped.hip", "qlr_grouped_fwd.hip", "qlr_grouped_bwd.hip", "qlr_grouped_grad.hip", "qlr_i8.hip"]


def compiled(path, *flags):
    cmd = [build.hipcc(), *build.COMMON, "-S", *flags, "--cuda-device-only", path, "-o", "-"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return res.stdout


def absolute_and_static(path):
    """(kernels that read LDS at absolute addresses, those of them with static LDS)"""
    ir, asm = compiled(path, "-emit-llvm"), compiled(path)
    static = {m[1]: int(m[2]) for m in
              re.finditer(r"\.amdhsa_kernel (\S+)\n(?:(?!\.end_amdhsa_kernel)[^\n]*\n)*?\s*\.amdhsa_group_segment_fixed_size (\d+)", asm)}
    absolute = set()
    for m in re.finditer(r"^define [^\n]*amdgpu_kernel [^\n]*@(\S+?)\([^\n]*\n(.*?)^}", ir, re.M | re.S):
        if re.search(r"inttoptr[^\n]*addrspace\(3\)", m[2]):
            absolute.add(m[1])
    assert static and absolute <= set(static)
    return absolute, {k for k in absolute if static[k] != 0}


def test_absolute_addresses_and_static_lds_do_not_meet():
    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        got = dict(zip(SOURCES, ex.map(lambda s: absolute_and_static(os.path.join(build.CSRC, s)), SOURCES)))
    assert all(not bad for _, bad in got.values()), got
    assert all("k_grouped_few" in k for a, _ in got.values() for k in a)
    assert len(got["qlr_grouped.hip"][0]) == 12  # four code widths, three shapes


def test_a_static_variable_is_found(tmp_path):
    """The same kernels with a static LDS variable put into one of them."""
    with open(os.path.join(build.CSRC, "qlr_grouped.hip")) as f:
        text = f.read()
    at = "  extern __shared__ uint32_t smem[];\n"
    assert text.count(at) == 1
    path = tmp_path / "qlr_grouped.hip"
    path.write_text(text.replace(at, at + "  __shared__ volatile int one;\n  one = 1;\n"))
    absolute, bad = absolute_and_static(str(path))
    assert len(bad) == len(absolute) == 12
