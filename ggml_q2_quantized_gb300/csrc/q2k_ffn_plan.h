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

// The most tiles of `rows` tokens that M tokens in `segments` segments have: every
// segment's last one may be a token's.
inline int segment_tiles(int M, int segments, int rows) {
    const int last = std::min(M, segments);
    return last + (M - last) / rows;
}

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

// The same for M tokens in `experts` segments of unknown lengths, each with matrices of
// its own: a token tile belongs to one segment, so there are at most M / x_rows tiles
// and one more for each segment that has tokens.  The kernel reads how many there are;
// all are whole.  Tokens per tile: a stage takes as long for 128 tokens as for fewer
// (the decode bounds it), and 0.7 of the time of 256 tokens; a segment of the mean
// length and its last tile, half full, then cost
//   (mean / x_rows + 1/2, at least 1) * (x_rows == 256 ? 1 : 0.7);
// of equal ones the narrower tile, which reads fewer rows that are not its segment's.
inline Plan make_segment_plan(int M, int rows, int tile_rows, int quads, int experts) {
    Plan best = {};
    double best_cost = 0;
    const double mean = static_cast<double>(M) / std::min(M, experts);
    for (int x_rows : {32, 64, 128, 256}) {
        const double cost = std::max(1.0, mean / x_rows + 0.5) * (x_rows == 256 ? 1.0 : 0.7);
        if (best_cost != 0 && cost >= best_cost) continue;
        best_cost = cost;
        best.x_rows = x_rows;
    }
    best.ctas = best.x_rows == 256 ? 2 : 1;
    const int row_tiles = (rows + tile_rows - 1) / tile_rows;
    best.row_units = (row_tiles + best.ctas - 1) / best.ctas;
    best.tiles = best.row_units * segment_tiles(M, experts, best.x_rows);
    best.whole = best.tiles;
    const int most = kPlanSms / best.ctas;
    best.workers = std::min(best.tiles, most);
    // a cluster divides a tile's K while every tile still has a worker of its own
    best.parts = std::max(1, std::min({kMaxParts / best.ctas, quads, most / best.tiles}));
    return best;
}

// ---- tokens in segments --------------------------------------------------------
// The offsets are data of the GPU that no call has seen: whatever they are, what follows
// gives tokens of the M, segments that there are, and no more tiles than there is room for.

Q2K_BOTH int held(int v, int least, int most) { return v < least ? least : v > most ? most : v; }

struct Tokens {
    int lo, hi;  // 0 <= lo <= hi <= M
};
// Those of segment e: [offsets[e], offsets[e + 1]).
Q2K_BOTH Tokens segment_tokens(const int* offsets, int e, int M) {
    Tokens t;
    t.lo = held(offsets[e], 0, M);
    t.hi = held(offsets[e + 1], t.lo, M);
    return t;
}
Q2K_BOTH int tiles_of(Tokens t, int rows) { return (t.hi - t.lo + rows - 1) / rows; }

struct TableEntry {
    int segment, first, tokens;
};
// Tile t of the table, t < begins[segments]: the last segment whose tiles begin at t or
// before has it.  begins: for each segment the tiles before it, held at the room there is;
// then their count, held the same.
Q2K_BOTH TableEntry table_entry(const int* begins, const int* offsets, int segments, int M, int rows, int t) {
    int a = 0, b = segments;
    while (b - a > 1) {
        const int mid = (a + b) / 2;
        if (begins[mid] <= t) a = mid;
        else b = mid;
    }
    const Tokens tokens = segment_tokens(offsets, a, M);
    TableEntry entry;
    entry.segment = a;
    entry.first = tokens.lo + (t - begins[a]) * rows;
    entry.tokens = held(tokens.hi - entry.first, 0, rows);
    return entry;
}

// The segment of a token that a warp looks for: its lanes found part `part` of `each`
// offsets, the last that begins at the token or before (-1: none), and `before` of that
// part's offsets there.  -1: no segment's.
Q2K_BOTH int segment_found(int part, int each, int before, int segments) {
    const int e = part * each + before - 1;
    return part >= 0 && e >= 0 && e < segments ? e : -1;
}

// ---- the gradient of a projection's activation ---------------------------------

// A lane of the kernel that forms a projection's dz has the kGradEach columns from n on, of
// rows of N values that lie one behind the other.  How many of them are the row's: in rows
// of whole words all or none, so that a lane reads a word or nothing.  (Its rows of the
// workspace are longer, up to a multiple of eight: with N = 4 mod 8 a lane begins where
// the row ends.)
constexpr int kGradEach = 4;
Q2K_BOTH int grad_inside(int n, int N) { return N - n >= kGradEach ? kGradEach : N > n ? N - n : 0; }

#undef Q2K_BOTH

}  // namespace q2k
