"""The sizes of test_gpu_gated_accumulate.py reach every tile of the weights' gradients, with and without ranges of
rows, by the library's own rule, compiled for the host."""
import os
import shutil
import subprocess

import pytest

from dense16_accumulate_cases import ACCUMULATE

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_expert_02_amd", "csrc")
MAIN = """#include <cstdio>
#include "dense16_rule.hpp"
int main() {
  long long M, H, I;
  while (scanf("%lld %lld %lld", &M, &H, &I) == 3) {
    const auto p = moe::d16::plan_of(moe::d16::DW, I, H, M);
    printf("%d %d\\n", p.bm, p.splits);
  }
}
"""


def test_every_tile_is_reached(tmp_path):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host compiler")
    (tmp_path / "main.cpp").write_text(MAIN)
    exe = str(tmp_path / "rule")
    subprocess.run([cxx, "-std=c++17", "-Wall", "-I", CSRC, str(tmp_path / "main.cpp"), "-o", exe], check=True, timeout=60)
    out = subprocess.run([exe], input="".join("%d %d %d\n" % c for c in ACCUMULATE), capture_output=True, text=True, check=True, timeout=60).stdout
    got = {(int(bm), int(s) > 1) for bm, s in (line.split() for line in out.splitlines())}
    assert got == {(256, False), (256, True), (128, False), (128, True)}
    # the columns' sums: one workgroup up to 256 rows, several beyond; never the kernel of few rows
    assert min(c[0] for c in ACCUMULATE) > 128 and any(c[0] <= 256 for c in ACCUMULATE) and any(c[0] > 256 for c in ACCUMULATE)
