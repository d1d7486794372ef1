"""Which kernel of moe_mx_linear the tests' sizes reach, by the library's own rule,
compiled for the host: a change of the rule that leaves a kernel untested fails here."""
import os
import shutil
import subprocess

import pytest

import mx_linear_cases as C

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_expert_02_amd", "csrc")
KERNELS = ("SKINNY_8_1_1_LITE", "SKINNY_4_1_1_LITE", "SKINNY_8_1_1", "SKINNY_4_2_1", "SKINNY_4_1_2", "SKINNY_X_2_2",
           "TILE_LARGEST", "TILE_128_128", "TILE_64_128", "TILE_64_64")
MAIN = """#include <cstdio>
#include "mx_linear_rule.hpp"
int main() {
  using moe::mxl::Kernel;
  int f8, exact, M, N, K;
  while (scanf("%%d %%d %%d %%d %%d", &f8, &exact, &M, &N, &K) == 5) switch (moe::mxl::choose(f8, exact, M, N, K)) {
%s
  }
}
""" % "\n".join(f'    case Kernel::{k}: puts("{k}"); break;' for k in KERNELS)


@pytest.fixture(scope="module")
def chosen(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("rule")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror=switch", "-I", CSRC, str(d / "main.cpp"), "-o", str(d / "rule")],
                   check=True, timeout=60)

    def ask(fmt, exact, *shapes):
        lines = "".join(f"{int(fmt == 'mxfp8')} {int(exact)} {M} {N} {K}\n" for M, N, K in shapes)
        return subprocess.run([str(d / "rule")], input=lines, capture_output=True, text=True, check=True,
                              timeout=60).stdout.split()
    return ask


def test_largest_tiles(chosen):
    for fmt, shapes in C.LARGEST.items():
        assert chosen(fmt, False, *shapes) == ["TILE_LARGEST"] * len(shapes)


@pytest.mark.parametrize("fmt,exact", [("mxfp8", True), ("mxfp8", False), ("mxfp4", False)])
def test_other_kernels(chosen, fmt, exact):
    got = chosen(fmt, exact, *[c[1:] for c in C.OTHERS])
    assert got == [c[0] for c in C.OTHERS]
    assert set(got) == set(KERNELS) - {"TILE_LARGEST"}


def test_epilogues(chosen):
    for kernel, fmt, M, widths in C.EPILOGUE:
        assert widths[0] % 8 == 0 and widths[1] % 8 != 0
        assert chosen(fmt, False, *[(M, N, C.EPILOGUE_K) for N in widths]) == [kernel] * 2
    assert {(k, f) for k, f, _, _ in C.EPILOGUE} == {(k, f) for k in KERNELS if k.startswith("TILE") for f in C.LARGEST}


def test_exact_kernels(chosen):
    got = chosen("mxfp8", True, *[(M, N, C.EXACT_K) for _, M, N in C.EXACT])
    assert got == [c[0] for c in C.EXACT] and set(got) == set(KERNELS) - {"TILE_LARGEST"}
    assert "TILE_LARGEST" not in chosen("mxfp8", True, *C.LARGEST["mxfp8"])
