"""moe_gated_grad_problem.two_parts without a GPU: its values, the workspace it asks for, and the tiles that the sizes of
test_gpu_gated_parts.py reach."""
import os
import shutil
import subprocess

import pytest

from mixture_experts_expert_02_amd import binding as B
from test_dense16_cpu import call_grad, gated
from test_gpu_gated_parts import MANY

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_expert_02_amd", "csrc")
MAIN = """#include <cstdio>
#include "dense16_rule.hpp"
int main() {
  using namespace moe::d16;
  long long M, H, I;
  while (scanf("%lld %lld %lld", &M, &H, &I) == 3) {
    const auto x = plan_of(DX, M, H, parts_k(I)), w = plan_of(DW, I, H, parts_k(M));
    printf("%d %d %d %d\\n", x.bm, x.splits, w.bm, w.splits);
  }
}
"""


def grad(two_parts, **kw):
    return B.MoeGatedGradProblem(gated(**kw), kw.get("type", 0), 0, 0, 0, 0, two_parts)


@pytest.mark.parametrize("value", [2, -1])
def test_other_values_are_refused(value):
    assert call_grad(grad(value)) == B.MOE_EINVAL
    assert B.moe_gated_linear_backward_workspace_bytes(grad(value)) == 0


@pytest.mark.parametrize("M,I", [(64, 264), (200, 264), (5000, 1032)])
def test_the_workspace_holds_both_parts(M, I):
    one, two = [B.moe_gated_linear_backward_workspace_bytes(grad(v, M=M, I=I)) for v in (0, 1)]
    assert one >= 2 * M * I * 2 and two >= 2 * 2 * M * I * 2
    assert call_grad(grad(1, M=M, I=I), size=two - 1) == B.MOE_ENOSPC


def test_every_tile_is_reached(tmp_path):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host compiler")
    (tmp_path / "main.cpp").write_text(MAIN)
    exe = str(tmp_path / "rule")
    subprocess.run([cxx, "-std=c++17", "-Wall", "-I", CSRC, str(tmp_path / "main.cpp"), "-o", exe], check=True, timeout=60)
    sizes = [c for c in MANY if c[0] > 64]
    out = subprocess.run([exe], input="".join("%d %d %d\n" % c for c in sizes), capture_output=True, text=True, check=True, timeout=60).stdout
    rows = [list(map(int, line.split())) for line in out.splitlines()]
    every = {(256, False), (256, True), (128, False), (128, True)}
    assert {(r[0], r[1] > 1) for r in rows} == every and {(r[2], r[3] > 1) for r in rows} == every
