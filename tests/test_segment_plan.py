"""The plan of a product over tokens in segments, on the host: the room for tiles is what
any lengths need and no more, and the grid fits the GPU."""

import subprocess

import pytest

from ggml_q2_quantized_gb300 import build as q2k_build

HARNESS = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "q2k_ffn_plan.h"
using namespace q2k;
#define CHECK(c) do { if (!(c)) { std::printf("M %d segments %d rows %d: %s\n", M, E, rows, #c); return 1; } } while (0)

// The most tiles that lengths c_1 .. c_E >= 0 with sum <= M have: by dynamic programming
// over segments, best[m] the most of m tokens.
static int most(int M, int E, int rows) {
    std::vector<int> best(M + 1, 0);
    for (int e = 0; e < E; ++e) {
        std::vector<int> next(best);
        for (int m = 1; m <= M; ++m)
            for (int c = 1; c <= m; ++c) {
                const int t = best[m - c] + (c + rows - 1) / rows;
                if (t > next[m]) next[m] = t;
            }
        best = next;
    }
    return best[M];
}

int main() {
    for (int M = 1; M <= 24; ++M)
        for (int E : {1, 2, 3, 5, 30})
            for (int rows : {1, 2, 4, 7, 8}) CHECK(segment_tiles(M, E, rows) == most(M, E, rows));
    for (int M : {1, 5, 100, 513, 4096, 70000, 1 << 20})
        for (int E : {1, 2, 7, 64, 256, 4096})
            for (int rows : {1, 8, 127, 1000, 7168, 1 << 20})
                for (int tile_rows : {64, 128})
                    for (int quads : {1, 2, 8, 28, 4096}) {
                        const Plan p = make_segment_plan(M, rows, tile_rows, quads, E);
                        CHECK((p.x_rows == 256) == (p.ctas == 2) && p.x_rows >= 32 && p.x_rows <= 256);
                        CHECK(static_cast<long long>(p.row_units) * p.ctas * tile_rows >= rows);
                        CHECK(static_cast<long long>(p.row_units) * segment_tiles(M, E, p.x_rows) == p.tiles);
                        CHECK(p.tiles > 0 && p.whole == p.tiles && p.partial == 0 && p.counts == 0);
                        CHECK(p.workers >= 1 && p.workers * p.ctas * p.parts <= kPlanSms);
                        CHECK(p.ctas * p.parts <= kMaxParts && p.parts <= quads);
                        CHECK(p.parts == 1 || p.tiles == p.workers);
                    }
    return 0;
}
"""


def test_segment_plans(tmp_path):
    src = tmp_path / "plan.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "plan"
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", q2k_build.CSRC, str(src),
                    "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout


@pytest.mark.parametrize("call", ["linear", "route", "sort", "sort_backward", "combine",
                                  "combine_backward", "linear_backward"])
def test_the_compiled_module_declines_what_is_not_ordinary(call):
    torch = pytest.importorskip("torch")
    import ggml_q2_quantized_gb300 as q2k
    quick = q2k._quick()
    counts = {"linear": 10, "route": 2, "sort": 3, "sort_backward": 3, "combine": 5,
              "combine_backward": 5, "linear_backward": 7}
    n = counts[call]
    for args in ((None,) * n, (torch.zeros(2, 256),) * n, ("x",) * n, (3,) * n, (), (None,) * (n + 1)):
        assert getattr(quick, call)(*args) is None


def test_bind_experts_wants_its_addresses():
    pytest.importorskip("torch")
    import ggml_q2_quantized_gb300 as q2k
    quick = q2k._quick()
    with pytest.raises(TypeError):
        quick.bind_experts(1, 2)
    with pytest.raises(ValueError):
        quick.bind_experts(*range(1, 13), 0)
