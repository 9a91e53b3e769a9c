"""How the tensor-core kernel divides its work, on the host: every block of K of every
tile goes to one worker, a worker has two runs of cut tiles at most, and all who have a
run of a tile agree on who they are.  And the plans that the GPU tests count on."""

import random
import subprocess

import pytest

from ggml_q2_quantized_gb300 import build as q2k_build

HARNESS = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "q2k_ffn_plan.h"
using namespace q2k;

#define CHECK(c) do { if (!(c)) { std::printf("M %d rows %d of %d quads %d: %s\n", M, rows, tile_rows, quads, #c); return 1; } } while (0)

static int check(int M, int rows, int tile_rows, int quads) {
    const Plan p = make_plan(M, rows, tile_rows, quads);
    CHECK(p.x_rows >= 32 && p.x_rows <= 256 && (p.x_rows == 256) == (p.ctas == 2));
    CHECK(p.row_units * p.ctas * tile_rows >= rows && (p.row_units - 1) * p.ctas * tile_rows < rows);
    CHECK(p.tiles == p.row_units * ((M + p.x_rows - 1) / p.x_rows));
    CHECK(p.workers * p.ctas * p.parts <= kPlanSms && p.ctas * p.parts <= kMaxParts);
    CHECK(p.parts == 1 || (p.tiles == p.workers && p.whole == p.tiles && p.parts <= quads));
    CHECK((p.partial != 0) == (p.whole < p.tiles) && (p.counts != 0) == (p.partial != 0));
    if (p.partial) {
        CHECK(p.partial >= static_cast<size_t>(2) * p.workers * p.ctas * p.x_rows * kPlanRows * 4);
        CHECK(p.counts >= static_cast<size_t>(p.tiles - p.whole) * p.ctas * 4);
        CHECK(p.whole >= p.workers && p.whole % p.workers == 0);
    }
    std::vector<unsigned char> seen(static_cast<size_t>(p.tiles) * quads, 0);
    std::vector<int> runs(p.tiles, 0);
    Segment s;
    for (int w = 0; w < p.workers; ++w)
        for (int part = 0; part < p.parts; ++part) {
            const Work k = {w, p.workers, quads, p.tiles, p.whole, part, p.parts};
            int n = 0;
            for (; k.segment(n, s); ++n) {
                CHECK(s.tile >= 0 && s.tile < p.tiles && s.q0 >= 0 && s.q0 < s.q1 && s.q1 <= quads);
                CHECK((s.run >= 0) == (s.tile >= p.whole));
                CHECK(s.run < 2 && (s.run < 0 || s.run == n));
                for (int q = s.q0; q < s.q1; ++q) CHECK(seen[static_cast<size_t>(s.tile) * quads + q]++ == 0);
                if (s.run >= 0) {
                    int first = -1, last = -1;
                    k.sharers(s.tile, first, last);
                    CHECK(first <= w && w <= last);
                    CHECK(k.run_of(w, s.tile) == s.run);
                    ++runs[s.tile];
                }
            }
            CHECK(n == k.count() && n > 0);
        }
    for (unsigned char c : seen) CHECK(c == 1);
    for (int t = p.whole; t < p.tiles; ++t) {
        const Work k = {0, p.workers, quads, p.tiles, p.whole, 0, p.parts};
        int first = -1, last = -1;
        k.sharers(t, first, last);
        CHECK(runs[t] == last - first + 1);
    }
    std::printf("%d %d %d %d %d %d\n", p.x_rows, p.tiles, p.whole, p.workers, p.ctas, p.parts);
    return 0;
}

int main() {
    int M, rows, tile_rows, quads, bad = 0;
    while (std::scanf("%d %d %d %d", &M, &rows, &tile_rows, &quads) == 4) bad |= check(M, rows, tile_rows, quads);
    return bad;
}
"""


@pytest.fixture(scope="module")
def planner(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(HARNESS)
    exe = str(at / "plan")
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", q2k_build.CSRC, str(at / "plan.cpp"), "-o", exe], check=True)

    def plans(shapes):
        text = "".join("%d %d %d %d\n" % s for s in shapes)
        res = subprocess.run([exe], input=text, capture_output=True, text=True)
        assert res.returncode == 0, res.stdout[-500:]
        return [dict(zip(("x_rows", "tiles", "whole", "workers", "ctas", "parts"), map(int, line.split())))
                for line in res.stdout.splitlines()]

    return plans


def gated(m, n, k):
    return m, n, 64, k // 256


def lora(m, n, k):
    return m, n, 128, k // 256


def backward(m, n, k):
    return m, k, 128, 2 * (-(-n // 128) * 128) // 256


def test_every_block_goes_to_one_worker(planner):
    rng = random.Random(1)

    def size(hi):
        return max(1, round(2 ** rng.uniform(0, hi)))

    shapes = [f(size(12), size(14.5), 256 * size(6)) for f in (gated, lora, backward) for _ in range(700)]
    shapes += [f(m, n, k) for f in (gated, lora, backward) for m in (1, 32, 33, 64, 65, 128, 129, 256, 257, 512)
               for n in (1, 64, 65, 4096, 9728, 9792, 14336) for k in (256, 512, 4096, 16384)]
    plans = planner(shapes)
    assert len(plans) == len(shapes)
    # all forms occur
    assert {p["x_rows"] for p in plans} == {32, 64, 128, 256}
    for x in (32, 64, 128, 256):
        assert any(p["x_rows"] == x and p["whole"] < p["tiles"] for p in plans)
        assert any(p["x_rows"] == x and p["parts"] > 1 for p in plans)


# (what test_gpu_ffn_divided runs, and the form it is there for)
EXPECTED = [
    (gated, 20, 12000, 16384, 32, True), (gated, 40, 12000, 16384, 64, True),
    (gated, 100, 12000, 16384, 128, True), (gated, 1024, 5000, 14336, 256, True),
    (gated, 600, 5000, 4096, 256, False), (gated, 300, 300, 1024, 128, False),
    (lora, 1024, 6000, 14336, 256, True), (lora, 1024, 5000, 14336, 128, True), (lora, 512, 14336, 1024, 256, False),
    (lora, 600, 5000, 4096, 256, False), (lora, 300, 9800, 1024, 128, False),
    (backward, 2048, 14336, 4096, 256, True), (backward, 600, 14336, 4096, 128, True),
    (backward, 1000, 14000, 2816, 128, True), (backward, 200, 9800, 14336, 256, False),
]


# Few blocks left over, cut among many workers: adding a tile's many runs takes longer
# than the round it saves (backwards 600 tokens, 5000 x 4096: 109 us cut and 77 whole;
# 200 tokens, 9800 x 14336: 194 and 172).
WHOLE = [(backward, 600, 5000, 4096), (gated, 200, 9800, 14336), (gated, 256, 14336, 4096)]


def test_tiles_stay_whole_where_their_runs_would_be_many(planner):
    for (f, *shape), p in zip(WHOLE, planner([f(*shape) for f, *shape in WHOLE])):
        assert p["whole"] == p["tiles"], (f.__name__, shape, p)


def test_plans_that_the_gpu_tests_count_on(planner):
    for (f, m, n, k, x_rows, cut), p in zip(EXPECTED, planner([f(m, n, k) for f, m, n, k, *_ in EXPECTED])):
        assert (p["x_rows"], p["whole"] < p["tiles"]) == (x_rows, cut), (f.__name__, m, n, k, p)
