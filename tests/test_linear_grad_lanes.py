"""Which columns the lanes of the kernel that forms a projection's dz read, on the host: the
rows' values once each, and nothing behind the last one."""

import subprocess

from ggml_q2_quantized_gb300 import build as q2k_build

HARNESS = r"""
#include <cstdio>
#include <vector>
#include "q2k_ffn_plan.h"
using namespace q2k;
#define CHECK(c) do { if (!(c)) { std::printf("N %d lane at column %d: %s\n", N, n, #c); return 1; } } while (0)

int main() {
    const int M = 3;
    for (int N = 1; N <= 1100; ++N) {
        const int pitch = (N + 7) & ~7;  // of the workspace's rows
        std::vector<int> read(static_cast<size_t>(M) * N, 0);
        int n = 0;
        for (; n < pitch; n += kGradEach) {
            const int inside = grad_inside(n, N);
            CHECK(inside >= 0 && inside <= kGradEach && (inside == 0 || n + inside <= N));
            // rows of whole words are read by the word
            if (N % kGradEach == 0) CHECK(inside == 0 || inside == kGradEach);
            for (int m = 0; m < M; ++m)
                for (int e = 0; e < inside; ++e) {
                    const size_t at = static_cast<size_t>(m) * N + n + e;
                    CHECK(at < read.size() && read[at] == 0);
                    read[at] = 1;
                }
        }
        for (int r : read) CHECK(r == 1);
    }
    return 0;
}
"""


def test_lanes_read_the_row_and_no_more(tmp_path):
    src = tmp_path / "lanes.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "lanes"
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", q2k_build.CSRC, str(src),
                    "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout
