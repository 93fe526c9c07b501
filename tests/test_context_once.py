"""CPU: what the kernels set once per CUDA context (csrc/context_once.h), with a fake of the context and of the call."""
import os
import subprocess

from xnor_popcount_gemm_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include "context_once.h"

int main() {
    unsigned long long here = 0;
    bool known = true;
    int calls = 0, result = 0;
    auto id = [&](unsigned long long *v) { *v = here; return known; };
    auto set = [&] { ++calls; return result; };
    bt::ContextOnce once;
    auto run = [&] { const int e = once.run(id, set); std::printf("%d %d\n", e, calls); };
    result = 7;
    run();                        // fails: tried again
    result = 0;
    run();
    run();                        // set in context 0
    here = 1;
    run();                        // another device's context
    run();
    here = 0;
    run();                        // back: at most once more
    run();
    known = false;
    run();                        // contexts that cannot be told apart: every time
    run();
    return 0;
}
"""


def test_once_per_context(tmp_path):
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    assert [tuple(map(int, line.split())) for line in out if line] == [
        (7, 1), (0, 2), (0, 2), (0, 3), (0, 3), (0, 4), (0, 4), (0, 5), (0, 6)]


def test_no_kernel_attribute_is_set_once_for_the_process():
    """Every call that sets a kernel's attribute goes through it."""
    for name in os.listdir(build.CSRC):
        text = open(os.path.join(build.CSRC, name)).read()
        if "cudaFuncSetAttribute" in text:
            assert name == "bt_internal.h", name
