// How the tensor-core kernel of the feed-forward operators divides a product: the plan
// of a call, and which tiles and runs of K each worker takes.  Plain C++, for the
// kernel and for the host.
#pragma once

#include <algorithm>
#include <cstddef>

#ifdef __CUDACC__
#define Q2K_BOTH __host__ __device__ __forceinline__
#else
#define Q2K_BOTH inline
#endif

namespace q2k {

constexpr int kMaxParts = 8;   // of K (the largest portable cluster)
constexpr int kPlanSms = 152;  // the work is cut for the whole GPU, whatever the device
constexpr int kPlanRows = 128; // rows of a CTA's tile

// One worker's share of the product (a CTA, or a pair): first its runs of the cut
// tiles (two at most), then its whole tiles.
struct Segment {
    int tile, q0, q1;
    int run;  // -1: a whole tile; else which of the worker's runs
};
struct Work {
    int w, workers, quads, tiles, whole;
    int part, parts;  // of K, for the CTAs of a cluster
    // quads [begin(w), begin(w + 1)) of the cut tiles, counted through
    Q2K_BOTH int begin(int w) const {
        return static_cast<int>(static_cast<long long>(tiles - whole) * quads * w / workers);
    }
    Q2K_BOTH bool segment(int index, Segment& s) const {
        const int a0 = begin(w), a1 = begin(w + 1);
        int runs = 0;
        if (a1 > a0) {
            const int t0 = a0 / quads, t1 = (a1 - 1) / quads;
            runs = t1 - t0 + 1;
            if (index < runs) {
                s.tile = whole + t0 + index;
                s.q0 = index == 0 ? a0 - t0 * quads : 0;
                s.q1 = index == runs - 1 ? a1 - t1 * quads : quads;
                s.run = index;
                return true;
            }
        }
        s.tile = w + (index - runs) * workers;
        s.q0 = quads * part / parts;
        s.q1 = quads * (part + 1) / parts;
        s.run = -1;
        return s.tile < whole;
    }
    Q2K_BOTH int count() const {
        const int a0 = begin(w), a1 = begin(w + 1);
        return (a1 > a0 ? (a1 - 1) / quads - a0 / quads + 1 : 0) +
               (w < whole ? (whole - 1 - w) / workers + 1 : 0);
    }
    // The workers with a run of cut tile `tile`.
    Q2K_BOTH void sharers(int tile, int& first, int& last) const {
        const long long q = static_cast<long long>(tile - whole) * quads;
        const long long total = static_cast<long long>(tiles - whole) * quads;
        first = static_cast<int>(q * workers / total);
        while (first > 0 && begin(first) > q) --first;
        while (begin(first + 1) <= q) ++first;
        last = first;
        while (last + 1 < workers && begin(last + 1) < q + quads) ++last;
    }
    // Which of worker v's runs is of cut tile `tile`.
    Q2K_BOTH int run_of(int v, int tile) const {
        return tile - whole - begin(v) / quads;
    }
};

struct Plan {
    int x_rows, row_units, tiles, whole, workers, ctas, parts;
    size_t partial, counts;  // bytes of workspace
};

// rows: those of the product; quads: its K in blocks (backward: 256 weight rows).
// Tokens per tile: as few as hold them all up to 64.  Above, 128 or 256,
// whichever is expected to end first: a worker's stages times the time of a
// stage, about 1 : 0.7 for 256 and 128 tokens.
inline Plan make_plan(int M, int rows, int tile_rows, int quads) {
    Plan best = {};
    double best_cost = 0;
    for (int x_rows : {32, 64, 128, 256}) {
        if (x_rows < 128 && x_rows < M) continue;
        Plan p = {};
        p.x_rows = x_rows;
        p.ctas = x_rows == 256 ? 2 : 1;
        const int row_tiles = (rows + tile_rows - 1) / tile_rows;
        p.row_units = (row_tiles + p.ctas - 1) / p.ctas;
        p.tiles = p.row_units * ((M + x_rows - 1) / x_rows);
        const int most = kPlanSms / p.ctas;
        const int rounds = p.tiles / most;
        p.parts = 1;
        p.whole = p.tiles;
        p.workers = std::min(p.tiles, most);
        double cost;
        if (rounds == 0) {
            p.parts = std::max(1, std::min({kMaxParts / p.ctas, quads, most / p.tiles}));
            cost = static_cast<double>(quads) / p.parts + 1;
        } else {
            // whole tiles only, or what is left after full rounds of them cut
            // evenly (a quad for every worker at least).  Bringing the runs' sums
            // together costs about 15 quads, and what adding a tile's runs takes (by
            // four warps of one CTA: 6 quads for a run of 128 tokens, 7 of 256, whose
            // quads are longer) beyond the whole tiles that are multiplied meanwhile.
            // Whole and cut, us: backwards 2048 tokens, 14336 x 4096, 392 and 357; 1200
            // 367 and 260; 600, 5000 x 4096, 77 and 109; gated 100 tokens, 12000 x
            // 16384, 148 and 105; 14336 x 4096, 128 tokens 43 and 55, 256 56 and 87;
            // 200 tokens, 9800 x 14336, 172 and 194.
            const long left = static_cast<long>(p.tiles - rounds * most) * quads;
            const double uncut = static_cast<double>(quads) * ((p.tiles + most - 1) / most);
            const double runs = static_cast<double>(quads) * most / std::max(left, 1l) + 1;
            const double adding = runs * (x_rows == 256 ? 7 : x_rows / 21.0) - static_cast<double>(rounds) * quads;
            const double cut = static_cast<double>(p.tiles) * quads / most + 15 + std::max(0.0, adding);
            const bool cuts = left >= most && cut < uncut;
            if (cuts) p.whole = rounds * most;
            cost = cuts ? cut : uncut;
        }
        cost *= x_rows == 256 ? 1.0 : 0.7;
        if (best_cost == 0 || cost < best_cost) {
            best = p;
            best_cost = cost;
        }
        if (x_rows >= M) break;  // a wider tile would be empty columns
    }
    if (best.whole < best.tiles) {
        best.partial = static_cast<size_t>(2) * best.workers * best.ctas * best.x_rows * kPlanRows * 4;
        best.counts = (static_cast<size_t>(best.tiles - best.whole) * best.ctas * 4 + 255) & ~size_t(255);
    }
    return best;
}

#undef Q2K_BOTH

}  // namespace q2k
