"""Host-side test: calls from several host threads share no variable that they write without synchronisation.  A function's own
`static` that can change is an atomic; one outside functions is thread-local."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
VARIABLE = re.compile(r"^\s*static\s+(?!constexpr\b|const\b|inline\b|__device__|std::atomic<|thread_local\b)[\w:<>,* ]+?\s\w+\s*(=|;|\{)")


def test_statics_that_change_are_atomic():
    files = sorted(f for pat in ("*.hip", "*.cpp", "*.h") for f in glob.glob(os.path.join(ROOT, "quantized_base_fine_amd", "csrc", pat)))
    assert len(files) > 20
    bad = []
    for f in files:
        for i, line in enumerate(open(f), 1):
            if VARIABLE.match(line) and "(" not in line.split("=")[0]:
                bad.append(f"{os.path.basename(f)}:{i}: {line.strip()}")
    assert not bad, bad


def test_the_search_finds_one():
    for line in ("  static bool attr = false;", "    static int cus = 0;  // of the device", "static std::string last;"):
        assert VARIABLE.match(line), line
    for line in ("  static constexpr int kT = KT;", "  static const Levels none{};", "  static std::atomic<bool> attr{false};",
                 "  static __device__ void f(Quad& a) {"):
        assert not VARIABLE.match(line), line
