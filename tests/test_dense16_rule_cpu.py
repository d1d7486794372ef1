"""Which tiles and K ranges the tests' sizes of the dense 16-bit projections reach, by the library's own rule,
compiled for the host: a change of the rule that leaves a kernel untested fails here."""
import os
import shutil
import subprocess

import pytest

import dense16_cases as C

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_expert_02_amd", "csrc")
MODES = {"gated": 0, "dx": 1, "dw": 2, "lora": 3}
MAIN = """#include <cstdio>
#include "dense16_rule.hpp"
int main() {
  int mode; long long M, N, K, R;
  while (scanf("%d %lld %lld %lld %lld", &mode, &M, &N, &K, &R) == 5) {
    const auto p = moe::d16::plan_of(mode, M, N, K);
    printf("%d %d %zu %d %d\\n", p.bm, p.splits, p.part, moe::d16::shrink_frags(M, R), moe::d16::shrink_ranges(M, K, R));
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("rule")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-I", CSRC, str(d / "main.cpp"), "-o", str(d / "rule")], check=True, timeout=60)

    def run(mode, *sizes):
        lines = "".join(f"{MODES[mode]} {' '.join(map(str, s))}\n" for s in sizes)
        out = subprocess.run([str(d / "rule")], input=lines, capture_output=True, text=True, check=True, timeout=60).stdout
        return [tuple(map(int, l.split())) for l in out.splitlines()]
    return run


def sizes(mode):
    if mode == "lora":
        return [(M, N, K, R) for M, K, N, R, L in C.LORA + C.LORA_LARGE if M > 64]
    all_ = C.GATED + C.GATED_LARGE
    if mode == "gated":
        return [(M, I, H, 8) for M, H, I in all_ if M > 32]
    return [(M, H, I, 8) if mode == "dx" else (I, H, M, 8) for M, H, I in all_]


@pytest.mark.parametrize("mode", list(MODES))
def test_tests_reach_every_tile_with_and_without_ranges(ask, mode):
    got = {(bm, s > 1) for bm, s, *_ in ask(mode, *sizes(mode))}
    assert got == {(256, False), (256, True), (128, False), (128, True)}


def test_tests_reach_every_form_of_the_first_product(ask):
    ranks = {min(r for r in (16, 32, 64, 128, 256) if R <= r) for *_, R in sizes("lora")}
    assert ranks == {16, 32, 64, 128, 256}
    got = {(f, r > 1) for *_, f, r in ask("lora", *sizes("lora"))}
    assert got == {(1, True), (1, False), (2, True), (2, False)}


@pytest.mark.parametrize("mode", list(MODES))
def test_plans_are_sound(ask, mode):
    """Partial results as large as their ranges need; no range without stages; the largest sizes take no ranges."""
    every = [(M, N, K, 16) for M in (1, 33, 129, 1000, 8193, 1 << 20) for N in (1, 8, 255, 2049, 1 << 20) for K in (8, 64, 65, 4104, 1 << 20)]
    for (M, N, K, _), (bm, s, part, _, ranges) in zip(every, ask(mode, *every)):
        stages = -(-K // 64) * (2 if mode == "dx" else 1)
        planes = 2 if mode in ("gated", "dw") else 1
        assert bm in (128, 256) and 1 <= s <= 16 and (s == 1 or 4 * s <= stages) and 1 <= ranges <= 16
        assert part >= (s > 1) * s * planes * M * ((N + 7) // 8 * 8) * 4 and part <= 300e6
