"""The cut of a product's k units into runs (csrc/q4_mx_runs.cuh), compiled for
the host: every unit in one run, each found by its owner, at most as many parts
a tile as the accuracy counts, and the sharers that the costs ask for."""
from __future__ import annotations

import math
import os
import subprocess
from fractions import Fraction

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_bit_gemv_b200", "csrc")
PARTS = 64      # parts of a tile that the stated accuracy counts

PROGRAM = r"""
#include <cstdio>
#include "q4_mx_runs.cuh"

// tiles groups Ku whole join part: sharers, ctas, most parts of a tile, 1 if the runs hold every unit once
int main() {
    int tiles, groups, Ku, join, part;
    long long whole;
    while (std::scanf("%d %d %d %lld %d %d", &tiles, &groups, &Ku, &whole, &join, &part) == 6) {
        const q4::RunCost cost = q4::run_cost(whole, join, part, Ku);
        const q4::RunCut cut(tiles, groups, Ku, cost);
        bool good = cut.ctas >= 1 && cut.ctas <= groups && cut.start(0) == 0 && cut.start(cut.ctas) == tiles * Ku;
        for (int c = 0; c < cut.ctas && good; ++c) {
            const int a = cut.start(c), b = cut.start(c + 1);
            good = a <= b && (b > a || tiles == 0);
            for (int v = a; v < b && good; v += b - a > 9 ? (b - a) / 9 : 1) good = cut.owner(v) == c;
            if (b > a) good = good && cut.owner(b - 1) == c;
        }
        int most = 0;
        for (int t = 0; t < tiles; ++t) {
            const int n = cut.owner((t + 1) * Ku - 1) - cut.owner(t * Ku) + 1;
            if (n > most) most = n;
        }
        std::printf("%d %d %d %d\n", cost.sharers, cut.ctas, most, good ? 1 : 0);
    }
}
"""


def _cases():
    """Sizes as q4_mx_gemm.cu makes them: CTAs or pairs, ns a k block, one or
    two k blocks a unit, tokens a tile."""
    for groups, block, unit, tokens in ((148, 190, 2, 8), (148, 190, 2, 16), (148, 190, 2, 32), (148, 270, 1, 64), (74, 370, 1, 72),
                                        (74, 370, 1, 120), (132, 270, 1, 40)):
        for Kb in (1, 2, 3, 7, 16, 32, 33, 64, 112, 441, 1000, 8192):
            for tiles in (0, 1, 2, 3, 5, 8, 16, 31, 32, 37, 73, 74, 75, 100, 147, 148, 149, 300, 1001):
                yield tiles, groups, -(-Kb // unit), Kb * block, 2000 + 70 * tokens, 300 + 14 * tokens


@pytest.fixture(scope="module")
def results(tmp_path_factory):
    d = tmp_path_factory.mktemp("runs")
    src, exe = d / "runs.cpp", d / "runs"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    cases = list(_cases())
    res = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stderr
    lines = [tuple(map(int, line.split())) for line in res.stdout.splitlines()]
    assert len(lines) == len(cases)
    return list(zip(cases, lines))


def test_runs_hold_every_unit_once(results):
    assert all(good == 1 for _, (_, _, _, good) in results)


def test_parts_of_a_tile(results):
    assert max(most for _, (_, _, most, _) in results) <= PARTS


def test_sharers_by_their_costs(results):
    for (tiles, groups, Ku, whole, join, part), (sharers, ctas, _, _) in results:
        assert sharers == min(max(math.isqrt(whole // part), 1), Ku)
        want = max(min(groups, tiles * Ku), 1)
        if 0 < tiles < groups:
            want = min(want, tiles * sharers)
            n = Fraction(want, tiles)
            if whole <= whole / n + join + part * n:
                want = tiles
        assert ctas == want


def test_the_kernel_cuts_in_whole_numbers():
    text = open(os.path.join(CSRC, "q4_mx_gemm.cu")).read()
    body = text[text.index("struct Runs {"):]
    body = body[:body.index("\n};\n")]
    assert "RunCut cut" in body and "float" not in body and "sqrt" not in body
