"""The tiles of tokens in segments from offsets of any values, on the host: the functions
that the kernels use never leave the tokens, the segments or the table's room, and
ascending offsets give every token of a segment once."""

import subprocess

from ggml_q2_quantized_gb300 import build as q2k_build

HARNESS = r"""
#include <algorithm>
#include <climits>
#include <cstdio>
#include <random>
#include <vector>
#include "q2k_ffn_plan.h"
using namespace q2k;
#define CHECK(c) do { if (!(c)) { std::printf("case %d M %d segments %d rows %d: %s\n", test, M, E, rows, #c); return 1; } } while (0)

static int test = 0;

// As the table's kernel: `threads` segments at a time, sums of those within 32 bits.
static int check(const std::vector<int>& offsets, int M, int rows, int threads, bool ascending) {
    const int E = static_cast<int>(offsets.size()) - 1, capacity = segment_tiles(M, E, rows);
    std::vector<int> begins(E + 1);
    long long carry = 0;
    for (int e0 = 0; e0 < E; e0 += threads) {
        long long sum = carry;
        for (int e = e0; e < E && e < e0 + threads; ++e) {
            const Tokens t = segment_tokens(offsets.data(), e, M);
            CHECK(0 <= t.lo && t.lo <= t.hi && t.hi <= M);
            begins[e] = static_cast<int>(sum < capacity ? sum : capacity);
            sum += tiles_of(t, rows);
            CHECK(sum <= INT_MAX);
        }
        carry = sum < capacity ? sum : capacity;
        if (ascending) CHECK(sum <= capacity);
    }
    begins[E] = static_cast<int>(carry);
    std::vector<unsigned char> seen(ascending ? M : 0, 0);
    for (int t = 0; t < begins[E]; ++t) {
        const TableEntry x = table_entry(begins.data(), offsets.data(), E, M, rows, t);
        CHECK(x.segment >= 0 && x.segment < E);
        CHECK(x.tokens >= 1 && x.tokens <= rows && x.first >= 0 && x.first <= M - x.tokens);
        if (!ascending) continue;
        CHECK(x.first >= offsets[x.segment] && x.first + x.tokens <= offsets[x.segment + 1]);
        for (int m = x.first; m < x.first + x.tokens; ++m) CHECK(seen[m]++ == 0);
    }
    for (int m = 0; m < static_cast<int>(seen.size()); ++m)
        CHECK(seen[m] == (m >= offsets[0] && m < offsets[E]));
    // a token's segment, as a warp finds it
    const int each = (E + 32) / 32, step = M > 300 ? M / 300 : 1;
    for (int m = 0; m < M; m += step) {
        int part = -1, before = 0;
        for (int lane = 0; lane < 32; ++lane) part += lane * each <= E && offsets[lane * each] <= m;
        if (part >= 0)
            for (int j = 0; j < each; ++j) before += part * each + j <= E && offsets[part * each + j] <= m;
        const int e = segment_found(part, each, before, E);
        CHECK(e >= -1 && e < E);
        if (!ascending) continue;
        CHECK(e < 0 ? m < offsets[0] || m >= offsets[E] : offsets[e] <= m && m < offsets[e + 1]);
    }
    ++test;
    return 0;
}

int main() {
    std::mt19937 rng(1);
    auto below = [&](int n) { return static_cast<int>(rng() % static_cast<unsigned>(n)); };
    for (int M : {1, 2, 7, 33, 300, 5000, 1 << 20})
        for (int E : {1, 2, 3, 31, 32, 33, 300, 1500, 4096})
            for (int rows : {1, 8, 32, 256})
                for (int threads : {256, 1024}) {
                    if (static_cast<long long>(M) * E > (1 << 22) && threads == 256) continue;
                    std::vector<int> o(E + 1);
                    // ascending, with empty segments and tokens before and behind
                    for (int& v : o) v = below(M + 1);
                    std::sort(o.begin(), o.end());
                    if (check(o, M, rows, threads, true)) return 1;
                    for (int& v : o) v = o[0];
                    o[E] = M;
                    if (check(o, M, rows, threads, true)) return 1;
                    // descending
                    for (int e = 0; e <= E; ++e) o[e] = M - static_cast<int>(static_cast<long long>(M) * e / E);
                    if (check(o, M, rows, threads, false)) return 1;
                    // overlapping: all tokens again and again
                    for (int e = 0; e <= E; ++e) o[e] = e & 1 ? M : 0;
                    if (check(o, M, rows, threads, false)) return 1;
                    for (int e = 0; e <= E; ++e) o[e] = e & 1 ? INT_MAX : INT_MIN;
                    if (check(o, M, rows, threads, false)) return 1;
                    // negative, past the end, and anything
                    for (int& v : o) v = -1 - below(M);
                    if (check(o, M, rows, threads, false)) return 1;
                    for (int& v : o) v = M + below(M);
                    if (check(o, M, rows, threads, false)) return 1;
                    for (int& v : o) v = below(3 * M) - M;
                    if (check(o, M, rows, threads, false)) return 1;
                    for (int& v : o) v = static_cast<int>(rng());
                    if (check(o, M, rows, threads, false)) return 1;
                }
    return 0;
}
"""


def test_table_of_any_offsets(tmp_path):
    src = tmp_path / "table.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "table"
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", q2k_build.CSRC, str(src),
                    "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout
