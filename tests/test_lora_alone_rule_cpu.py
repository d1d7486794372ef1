"""The sizes of test_gpu_lora_alone.py reach every way through the adapters' second product, by the library's own rules,
compiled for the host."""
import os
import shutil
import subprocess

import pytest

from lora_alone_cases import ALONE

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_expert_02_amd", "csrc")
MAIN = """#include <cstdio>
#include "dense16_rule.hpp"
int main() {
  long long M, K; int R;
  while (scanf("%lld %lld %d", &M, &K, &R) == 3)
    printf("%d %d\\n", moe::d16::expand_frags(M), moe::d16::shrink_ranges(M, K, R));
}
"""


def test_every_way_is_reached(tmp_path):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host compiler")
    (tmp_path / "main.cpp").write_text(MAIN)
    exe = str(tmp_path / "rule")
    subprocess.run([cxx, "-std=c++17", "-Wall", "-I", CSRC, str(tmp_path / "main.cpp"), "-o", exe], check=True, timeout=60)
    lines = "".join(f"{M} {K} {R}\n" for M, K, _, R, _ in ALONE)
    out = subprocess.run([exe], input=lines, capture_output=True, text=True, check=True, timeout=60).stdout
    got, most = set(), 0
    for (M, _, _, R, _), line in zip(ALONE, out.splitlines()):
        frags, ranges = map(int, line.split())
        most = max(most, ranges)
        got.add((frags, ranges > 1, R > 64))
    assert got == {(f, r, k) for f in (1, 4) for r in (False, True) for k in (False, True)}
    assert most == 16
