"""The host-side plan of the experts kernel, compiled as plain C++ (no GPU needed)."""
import os
import shutil
import subprocess
from fractions import Fraction
from math import comb

import pytest

from conftest import ROOT

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "moe_plan.cuh"
int main(int argc, char **argv) {
    for (int i = 1; i + 4 < argc; i += 5) {
        const int M = atoi(argv[i]), E = atoi(argv[i + 1]), k = atoi(argv[i + 2]), H = atoi(argv[i + 3]), F = atoi(argv[i + 4]);
        const double c = nf4::moe_expected_chunks(M, E, k);
        std::printf("%.17g %d\n", c, nf4::pick_moe_group(c, F / 32, (H / 64 + 1) / 2, H / 64, (F / 64 + 1) / 2, 148));
    }
}
"""

CASES = [(1, 64, 8, 2048, 1024), (4, 8, 2, 5120, 13824), (16, 64, 6, 2048, 1408), (37, 32, 4, 4096, 1792),
         (64, 8, 8, 2048, 1024), (64, 8, 2, 2048, 1024), (1, 1, 1, 64, 64), (64, 1, 1, 128, 128), (64, 256, 16, 64, 64),
         (64, 17, 16, 256, 256), (9, 2, 2, 448, 704), (33, 3, 2, 1088, 576), (28, 2, 2, 576, 4160), (51, 2, 2, 704, 3584)]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    csrc = os.path.join(ROOT, "bit_nf4_quantized_05_b200", "csrc")
    cc = subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I" + csrc, str(d / "plan.cpp"), "-o",
                         str(d / "plan")], capture_output=True, text=True)
    assert cc.returncode == 0, cc.stderr
    run = subprocess.run([str(d / "plan")] + [str(v) for c in CASES for v in c], capture_output=True, text=True, timeout=60)
    rows = [line.split() for line in run.stdout.splitlines()]
    assert len(rows) == len(CASES)
    return [(float(c), int(g)) for c, g in rows]


def test_expected_chunks_count_an_experts_tokens_in_eights(plan):
    """Against the binomial distribution in exact fractions: 64 tokens at all of 8
    experts are 64 chunks, not 8."""
    for (M, E, k, _, _), (got, _) in zip(CASES, plan):
        p = Fraction(k, E)
        want = E * sum(comb(M, n) * p ** n * (1 - p) ** (M - n) * ((n + 7) // 8) for n in range(M + 1))
        assert abs(got - float(want)) <= 1e-12 * float(want), (M, E, k)
    assert plan[4][0] == 64.0


def test_group_sizes(plan):
    """The group sizes that were fastest when measured (within 1.5%)."""
    fast = {(1, 64, 8, 2048, 1024): (8,), (4, 8, 2, 5120, 13824): (8,), (16, 64, 6, 2048, 1408): (4,),
            (37, 32, 4, 4096, 1792): (4, 8), (64, 8, 8, 2048, 1024): (4, 8), (64, 8, 2, 2048, 1024): (8,),
            (28, 2, 2, 576, 4160): (8,), (51, 2, 2, 704, 3584): (8,)}
    for c, (_, g) in zip(CASES, plan):
        assert g in fast.get(c, (4, 8, 16)), (c, g)
