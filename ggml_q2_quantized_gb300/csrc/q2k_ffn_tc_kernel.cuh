// Many tokens times Q2_K weights on the tensor cores (tcgen05): the gated
// feed-forward block, its backward product, and a projection with low-rank
// adapters.
//
// A CTA computes 128 rows of a product x up to 256 tokens: 16 warps decode Q2_K
// blocks into shared or tensor memory (the MMA's A operand), token stages of 64 K
// arrive by TMA in the 128-byte-swizzled layout that the MMA reads (the B operand;
// f32 tokens come from a bf16 image that a prepass writes in that layout), and f32
// sums build up in tensor memory, in two sets: four warps bring one tile's sums
// out while the next tile is multiplied into the other (gated, 512 tokens x 14336
// x 4096: a tile's set-up and epilogue took 8 of its 33 us before).
//
// Gated: the 128 rows are 64 rows of Wg and the same 64 rows of Wu, so one tile
// holds both projections of its outputs and the MMAs run as for one matrix; g
// and u then meet in shared memory, where the activation and the product are
// taken before anything is stored.
//
// Backward: dx = [dg du] [Wg; Wu], a product over the weights' rows.  A tile's
// 128 rows are half a block of columns (k), a stage is 64 weight rows.  A thread
// decodes a weight row as above (one table serves 16 codes) and stores it as
// stored, k running, which is the MMA's A operand "MN-major": the transposition
// costs nothing.  (Transposing the codes first, so that a lane could write its
// own column to tensor memory, took more instructions than the stores it saved.)
//
// Work split, K in blocks (backward: in 256 weight rows):
// - fewer tiles than half of the workers (CTAs, or pairs, that the GPU holds): a
//   cluster of up to eight CTAs divides a tile's K; the parts' sums meet through
//   distributed shared memory, each part bringing out a share of the tokens;
// - more tiles than workers: whole tiles go to the workers in turn, and what is
//   left over, less than a tile each, is cut into equal runs of K, so that all
//   end together.  The runs come first: their sums go to the workspace, the CTA
//   that finishes last adds them, in the order of K whoever that is, and all of
//   that happens while whole tiles are multiplied.  No CTA waits for another.
//   (2048 tokens backwards, 14336 x 4096: 128 tiles for 76 pairs, the whole call 357
//   us against 392 in two rounds.  Cutting without whole tiles behind it, or into
//   many runs, exposes the adding.)
//
// What bounds it: at 256 tokens a tile the MMAs and the shared memory that feeds
// them (per stage and SM 32 KB of operands read, 32 KB written: 512 of about 740
// clocks at 128 bytes a clock; 0.38 us a stage of 64 K, where a plain bf16 product
// at the measured peak takes 0.34); below, the decode (0.33 us a stage at 128
// tokens).
//
// Every wait is bounded (about a second); on time-out the kernel records a bit
// in the device error word, drains its MMAs, frees TMEM and returns.
#pragma once

#include <algorithm>
#include <atomic>
#include <cstring>

#include "q2k_ffn_tc.cuh"

namespace q2k {

namespace {

// This file's error word (a word of its own in each file, since a pointer to a shared
// one costs a register that the kernel does not have: 0.5 % of its time).
__device__ unsigned int g_tc_error;
const bool g_tc_error_known = add_tc_error_word(&g_tc_error);

using namespace tc;

constexpr int kDecWarps = 16;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kMmaWarp = kDecWarps, kWaitWarp = kDecWarps + 1, kWWarp = kDecWarps + 2,
              kXWarp = kDecWarps + 3, kEpiWarp0 = kDecWarps + 4;  // (a multiple of 4)
constexpr int kThreads = 32 * (kDecWarps + 8);

static_assert(kRows == kPlanRows, "a tile's rows");
constexpr int kABytes = kStageK * kRows * 2;  // a decoded stage in shared memory
// Sums of 32 tokens on their way out: token c, row r at word 132 c + r (132:
// lanes that read two tokens apart fall on different banks).
constexpr int kSumPitch = kRows + 4;
constexpr int kChunk = 32;

// Tiles of kX tokens.
// 256: two CTAs of a cluster (neighbouring row tiles) form one MMA of 256 rows
// x 256 tokens, issued by one thread of the first (cta_group::2).  Each holds
// half of the tokens' stage, so a stage is half as large and crosses from L2
// once per pair.
// 128 and fewer: the decode bounds, and narrow MMAs that read A from shared
// memory take as long as wide ones (100 clocks each, measured), so decoded
// weights go to tensor memory (not backward, where they would have to be
// transposed).  (14336 x 4096, 64 tokens: 52 us against
// 55 with A in shared memory; 40 since one elected thread issues the MMAs.)
template <int kX, bool kTma, Tc kMode>
struct Cfg {
    static constexpr bool kBack = kMode == Tc::kBackward;
    static constexpr bool kDuo = kX == 256;
    static constexpr int kCtas = kDuo ? 2 : 1;
    static constexpr bool kTmemA = !kBack && !kDuo;
    static constexpr int kHand = 2;                      // stages handed over at a time
    static constexpr int kHold = kX / kCtas;             // tokens of a stage in this CTA
    static constexpr int kXStage = kHold * kStageK * 2;
    // stages in flight, tokens and decoded weights alike (one release for both)
    static constexpr int kStages = kTmemA ? 8 : kX >= 128 ? 5 : kX == 64 ? 7 : 8;
    static constexpr int kGroupWarps = 4;  // decoders: four groups, a stage each in turn
    // (MMAs end in the order of their issue: a decoder's wait for those of stage
    // i - kStages by its barrier's parity is right because its wait before, for
    // stage i - 4 - kStages, covered i - 2 kStages)
    static constexpr uint32_t kAccCols = kX;             // a tile's sums; two sets
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kColA = 2 * kAccCols;      // 32 columns per decoded stage
    static_assert(kColA + (kTmemA ? 32 * kStages : 0) <= kTmemCols, "tensor memory");
    // raw slots: a block column of 128 weight rows, or (backward) of 64 for a
    // stage, without TMA only the 11 words of the half block that it needs
    static constexpr int kRawRows = kBack ? kStageK : kRows;
    static constexpr int kRawPitch = kTma || !kBack ? kBoxBytes : 44;
    // (forward without TMA maps of single rows: rows that no map covers beside them)
    static constexpr int kRawBytes = (kRawRows + (kTma || kBack ? 0 : 8)) * kRawPitch;
    static constexpr int kRaw = kBack ? (kTma ? 4 : 8) : kTmemA ? 4 : 2;
    static constexpr int kOffA = kStages * kXStage;
    static constexpr int kOffRaw = kOffA + (kTmemA ? 0 : kStages * kABytes);
    static constexpr int kOffSums = kOffRaw + kRaw * kRawBytes;
    // with adapters: 64 t for each token of a chunk; an id and whose for each of
    // the tile
    static constexpr int kOffT = kOffSums + kChunk * kSumPitch * 4;
    static constexpr int kOffIds = kOffT + (kMode == Tc::kLora ? kChunk * 64 * 4 : 0);
    // bars: x_full, a_full, peer_full, empty [kStages], raw_full, raw_empty
    //       [kRaw], acc_full, acc_empty [2], drain
    static constexpr int kNumBars = 4 * kStages + 2 * kRaw + 5;
    static constexpr int kOffBar = (kOffIds + (kMode == Tc::kLora ? kX * 8 : 0) + 7) & ~7;
    static constexpr int kOffMisc = kOffBar + 8 * kNumBars;
    static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory");
    static_assert(kOffA % 1024 == 0 && kOffRaw % 1024 == 0 && kOffSums % 16 == 0 && kOffT % 64 == 0 &&
                      kSumPitch * 32 * 4 % 64 == 0,
                  "alignment");
    // the last tile's sums, t and ids for all its tokens, take the rings' place
    static_assert(kX * (kSumPitch + (kMode == Tc::kLora ? 64 : 0)) * 4 <= kOffIds, "epilogue");
};

// A box of raw weights at (x, row): of one matrix, or (kSeg) of an expert's.
template <bool kSeg>
__device__ __forceinline__ void load_weights(uint32_t dst, const CUtensorMap* map, int x, int row, int expert,
                                             uint32_t bar) {
    if constexpr (kSeg) tma_load_3d(dst, map, x, row, expert, bar);
    else tma_load_2d(dst, map, x, row, bar);
}

struct TcMaps {
    // weights, 112-byte boxes of 64 or 128 rows (or of every fourth of those rows,
    // where only four rows together are a multiple of 16 bytes)
    CUtensorMap w0, w1;
    CUtensorMap x0, x1;  // tokens, boxes of kX rows x 64 (backward: dg and du)
};

// Where row r of a tile lies in a raw slot whose rows came four to a group: rows of
// one place in their group together; `word`: a row that no group covers, behind them.
template <int kSplit0>
__device__ __forceinline__ int raw_place(int r, bool word) {
    const int half = r / kSplit0, rr = r % kSplit0;
    return word ? kRows + 4 * half + (rr & 3) : kSplit0 * half + kSplit0 / 4 * (rr & 3) + (rr >> 2);
}

// The threads that bring a tile's sums out: the epilogue's four warps while the
// next tile is being multiplied, those and the decoders for the CTA's last tile.
// Warp w of a team has TMEM lanes (rows) 32 (w % 4) ..
struct Team {
    int thread, threads, barrier;
    __device__ __forceinline__ void sync() const {
        asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(threads) : "memory");
    }
};

__device__ __forceinline__ float ld_shared_f32(uint32_t at) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint2 ld_shared_pair(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
    return v;
}
__device__ __forceinline__ void st_shared_f32(uint32_t at, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

// The ids of a tile's tokens [lo, hi) (multiples of eight; -1 none or past `tokens`,
// -2 out of range), and whose each is, sorted by id within every `scope` of them
// (those without an adapter last): what add_adapters takes at a time then has few
// adapters in a group of eight (512 tokens of four adapters in any order, rank 64:
// 154 us in the order they came).  A token counts those before it.  For four warps,
// while the tile is multiplied.
template <int kX>
__device__ __forceinline__ void sort_tokens(int* id_buf, int* order, const TcArgs& p, int m, int tokens,
                                            int lo, int hi, int scope, int et) {
    constexpr int kEach = (kX + 127) / 128;
    int id[kEach], at[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int c = lo + et + 128 * u;
        id[u] = -1;
        if (c < min(tokens, hi)) {
            id[u] = p.ids[m + c];
            if (id[u] < -1 || id[u] >= p.n_adapters) id[u] = -2;
        }
        if (c < hi) order[c] = id[u];
    }
    asm volatile("bar.sync 2, 128;" ::: "memory");
    // (already in order: whole requests one after another)
    uint32_t back = 0;
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int c = lo + et + 128 * u;
        at[u] = c;
        if (c > lo && c < hi) back |= static_cast<uint32_t>(order[c - 1]) > static_cast<uint32_t>(id[u]);
    }
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t"
        "bar.red.or.pred p, 2, 128, p;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "+r"(back)::"memory");
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int c = lo + et + 128 * u;
        if (c >= hi || back == 0) break;
        const int first = lo + (c - lo) / scope * scope, end = min(first + scope, hi);
        const uint32_t key = static_cast<uint32_t>(id[u]);
        at[u] = first;
#pragma unroll 1
        for (int j = first; j < end; j += 4) {
            const uint4 k = *reinterpret_cast<const uint4*>(order + j);
            at[u] += (k.x < key || (k.x == key && j < c)) + (k.y < key || (k.y == key && j + 1 < c)) +
                     (k.z < key || (k.z == key && j + 2 < c)) + (k.w < key || (k.w == key && j + 3 < c));
        }
    }
    asm volatile("bar.sync 2, 128;" ::: "memory");
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int c = lo + et + 128 * u;
        if (c >= hi) break;
        id_buf[at[u]] = id[u];
        order[at[u]] = c;
    }
    asm volatile("bar.sync 2, 128;" ::: "memory");
}

// Adds s_a B_a t of each token's adapter to the sums of `count` tokens from m on:
// per 16 rows and eight tokens, one product (m16n8k16) for each adapter that
// occurs among them, B_a as stored and t split into two bf16 (16 bits); a token's
// sum takes only its own adapter's product.  Slot c is the token order[c] of `sums`
// and of m.  t comes through shared memory 64 values a token at a time, already
// split: the two bf16 of value pair j (hi, lo) of slot c at words 64 c + (2 j ^
// 8 (c % 4)), so that the eight tokens a warp reads together fall on different
// banks.  A warp has 16 rows at a time, and keeps B_a's fragments in registers from
// one token group to the next with the same adapter.  128 rows x 256 tokens at rank
// 64 take about 10 us: 3 of products, 3 of B's rows, the rest instructions around
// them (by pointers instead of shared addresses, with spills, 15).
__device__ __forceinline__ void add_adapters(float* sums, uint32_t* tbuf, const int* id_buf,
                                             const int* order, const TcArgs& p, int n0, int m, int count,
                                             const Team& team) {
    const int et = team.thread, lane = et & 31;
    const int g = lane >> 2, t = lane & 3;
    const int slots = (count + 7) & ~7;
    for (int r0 = 0; r0 < p.R; r0 += 64) {
        const int width = min(64, p.R - r0);  // a multiple of 8
        for (int base = et; base < 16 * slots; base += 4 * team.threads) {
            float4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = base + team.threads * u, r = 4 * (i & 15);
                v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if ((i >> 4) < slots && r < width && id_buf[i >> 4] >= 0)
                    v[u] = *reinterpret_cast<const float4*>(p.t + static_cast<size_t>(m + order[i >> 4]) * p.R + r0 + r);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = base + team.threads * u, c = i >> 4, r = 4 * (i & 15);
                if (c >= slots) break;
                uint4 w;
                w.x = pack_bf16(v[u].x, v[u].y);
                w.z = pack_bf16(v[u].z, v[u].w);
                w.y = pack_bf16(v[u].x - __uint_as_float(w.x << 16),
                                v[u].y - __uint_as_float(w.x & 0xFFFF0000u));
                w.w = pack_bf16(v[u].z - __uint_as_float(w.z << 16),
                                v[u].w - __uint_as_float(w.z & 0xFFFF0000u));
                // (an infinity is its first part alone: the other would be NaN, and is 2^120)
                w.y = min_bf16x2(w.y, 0x7B807B80u);
                w.w = min_bf16x2(w.w, 0x7B807B80u);
                *reinterpret_cast<uint4*>(tbuf + 64 * c + (r ^ (8 * (c & 3)))) = w;
            }
        }
        team.sync();
        // row tile % 8 of warp % 8; the team's other warps take other tokens
        const int warp = et >> 5, warps = team.threads >> 5;
        const int sets = max(1, warps >> 3);
        // (shared addresses: half the registers of pointers)
        const uint32_t sums_at = smem_u32(sums) + 4 * g;
        const uint32_t ids_at = smem_u32(id_buf), order_at = smem_u32(order);
        // this lane's pair of step q and of the eight values on, word (16 q + 2 t) ^
        // 8 (g % 4) and that ^ 8
        const uint32_t t_at = smem_u32(tbuf) + 256 * g + 8 * t + 32 * (g & 1), t_swap = 64 * ((g >> 1) & 1);
#pragma unroll 1
        for (int rt = warp & 7; rt < 8 && (warp >> 3) < sets; rt += min(warps, 8)) {
            const int n = n0 + 16 * rt + g;  // this lane's rows: n, n + 8
            int cur = -1;
            uint32_t b[4][4];
#pragma unroll 1
            for (int c0 = 8 * (warp >> 3); c0 < slots; c0 += 8 * sets) {
                const int id = static_cast<int>(ld_shared_u32(ids_at + 4 * (c0 + g)));
                // the ids and tokens of the columns 2 t, 2 t + 1 whose sums this lane holds
                const uint2 ids2 = ld_shared_pair(ids_at + 4 * (c0 + 2 * t));
                const uint2 tokens = ld_shared_pair(order_at + 4 * (c0 + 2 * t));
                const int id0 = static_cast<int>(ids2.x), id1 = static_cast<int>(ids2.y);
                const uint32_t s0 = sums_at + 4 * (tokens.x * kSumPitch + 16 * rt);
                const uint32_t s1 = sums_at + 4 * (tokens.y * kSumPitch + 16 * rt);
                const uint32_t t_row = t_at + 256 * c0;
                if (id0 == -2) {
                    st_shared_f32(s0, 0.f);
                    st_shared_f32(s0 + 32, 0.f);
                }
                if (id1 == -2) {
                    st_shared_f32(s1, 0.f);
                    st_shared_f32(s1 + 32, 0.f);
                }
                unsigned todo = __ballot_sync(0xFFFFFFFFu, id >= 0);
                while (todo != 0) {
                    const int ad = __shfl_sync(0xFFFFFFFFu, id, __ffs(todo) - 1);
                    todo &= ~__ballot_sync(0xFFFFFFFFu, id == ad);
                    if (ad != cur) {
                        cur = ad;
                        const uint32_t* b0 = reinterpret_cast<const uint32_t*>(
                            p.b + (static_cast<size_t>(ad) * p.N + n) * p.R + r0) + t;
                        const uint32_t* b1 = b0 + 4 * p.R;  // eight rows on
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const bool in0 = 16 * q < width, in1 = 16 * q + 8 < width;
                            b[q][0] = n < p.N && in0 ? __ldg(b0 + 8 * q) : 0u;
                            b[q][1] = n + 8 < p.N && in0 ? __ldg(b1 + 8 * q) : 0u;
                            b[q][2] = n < p.N && in1 ? __ldg(b0 + 8 * q + 4) : 0u;
                            b[q][3] = n + 8 < p.N && in1 ? __ldg(b1 + 8 * q + 4) : 0u;
                        }
                    }
                    // (four chains of two products: one takes as long as dozens
                    // of other instructions to return)
                    float e[4][4] = {};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint2 u = make_uint2(0u, 0u), w = u;
                        if (id == ad && 16 * q < width) {
                            const uint32_t at = (q & 1 ? t_row - t_swap : t_row + t_swap) + 64 * q;
                            u = ld_shared_pair(at);
                            w = ld_shared_pair(at ^ 32u);
                        }
                        if (16 * q < width) {
                            mma_bf16_16816(e[q], b[q][0], b[q][1], b[q][2], b[q][3], u.x, w.x);
                            mma_bf16_16816(e[q], b[q][0], b[q][1], b[q][2], b[q][3], u.y, w.y);
                        }
                    }
                    float d[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) d[c] = (e[0][c] + e[1][c]) + (e[2][c] + e[3][c]);
                    if (id0 == ad) {
                        st_shared_f32(s0, ld_shared_f32(s0) + d[0]);
                        st_shared_f32(s0 + 32, ld_shared_f32(s0 + 32) + d[2]);
                    }
                    if (id1 == ad) {
                        st_shared_f32(s1, ld_shared_f32(s1) + d[1]);
                        st_shared_f32(s1 + 32, ld_shared_f32(s1 + 32) + d[3]);
                    }
                }
            }
        }
        team.sync();
    }
}

template <typename T>
__device__ __forceinline__ void store_pair(T* dst, float a, float b, int valid, bool vec);
template <>
__device__ __forceinline__ void store_pair(float* dst, float a, float b, int valid, bool vec) {
    if (vec) {
        *reinterpret_cast<float2*>(dst) = make_float2(a, b);
    } else {
        if (valid > 0) dst[0] = a;
        if (valid > 1) dst[1] = b;
    }
}
template <>
__device__ __forceinline__ void store_pair(__nv_bfloat16* dst, float a, float b, int valid, bool vec) {
    if (vec) {
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16(a, b);
    } else {
        if (valid > 0) dst[0] = __float2bfloat16_rn(a);
        if (valid > 1) dst[1] = __float2bfloat16_rn(b);
    }
}

__device__ __forceinline__ float4 load_cluster4(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .u32 ra;\n\tmapa.shared::cluster.u32 ra, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [ra];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

// Backward, non-TMA: the words of 64 weight rows that a stage needs (two of
// scales, eight of codes, d and dmin) packed into a raw slot, by the 128 threads
// of a decoder group.  Rows past N are zero (they decode to 0).
__device__ __forceinline__ void issue_raw_rows(const TcArgs& p, uint32_t dst, int stage, int expert,
                                               int block, int half, int tg) {
    const bool up = stage >= p.half_stages;
    const int n0 = kStageK * (up ? stage - p.half_stages : stage);
    const size_t row_bytes = static_cast<size_t>(p.K / kQK) * kBlockBytes;
    const uint8_t* w = (up ? p.w1 : p.w0) + static_cast<size_t>(expert) * p.N * row_bytes;
    for (int f = tg; f < kStageK * 11; f += 128) {
        const int r = f / 11, i = f - 11 * r;
        const int word = i < 2 ? 2 * half + i : i < 10 ? 4 + 8 * half + (i - 2) : 20;
        const bool ok = n0 + r < p.N;
        const uint8_t* src = w + (ok ? static_cast<size_t>(n0 + r) * row_bytes +
                                           static_cast<size_t>(block) * kBlockBytes + 4 * word
                                     : 0);
        cp_async_4(dst + 4 * f, src, ok ? 4u : 0u);
    }
    cp_async_commit();
}

// The 16 weights of a segment of one row at shift J: its four quant words -> bf16,
// k running.
template <int J>
__device__ __forceinline__ void decode_segment(const uint32_t (&q)[4], uint32_t sc, float d, float dmin,
                                               uint32_t (&o)[8]) {
    uint32_t lo, hi;
    weight_table(sc, d, dmin, lo, hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t sel = code_selectors<J>(q[e]);
        o[2 * e] = __byte_perm(lo, hi, sel);
        o[2 * e + 1] = __byte_perm(lo, hi, __umulhi(sel, 0x10000u));  // sel >> 16
    }
}

// Results of `count` tokens (m0 on) of a tile from their sums.
template <Tc kMode, typename T>
__device__ __forceinline__ void emit(const TcArgs& p, const float* sums, int n0, int rows, int m0,
                                     int count, const Team& team) {
    const int lane = team.thread & 31;
    const bool vec = (rows & 1) == 0;  // (n0 is even: pairs are aligned)
    // a warp takes a token at a time, a lane neighbouring rows
    for (int c = team.thread >> 5; c < count; c += team.threads >> 5) {
        const float* row = sums + c * kSumPitch + 2 * lane;
        const size_t at = static_cast<size_t>(m0 + c) * rows + n0 + 2 * lane;
        const int valid = rows - (n0 + 2 * lane);
        if constexpr (kMode == Tc::kGated) {
            if (valid <= 0) continue;
            const float2 g = *reinterpret_cast<const float2*>(row);
            const float2 u = *reinterpret_cast<const float2*>(row + kRows / 2);
            store_pair(static_cast<T*>(p.h) + at, act_value<sizeof(T) == 2>(g.x, p.act) * u.x,
                       act_value<sizeof(T) == 2>(g.y, p.act) * u.y, valid, vec);
            if (p.gate != nullptr) {
                store_pair(static_cast<T*>(p.gate) + at, g.x, g.y, valid, vec);
                store_pair(static_cast<T*>(p.up) + at, u.x, u.y, valid, vec);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float2 v = *reinterpret_cast<const float2*>(row + 64 * q);
                if (valid - 64 * q > 0)
                    store_pair(static_cast<T*>(p.y) + at + 64 * q, v.x, v.y, valid - 64 * q, vec);
            }
        }
    }
}

// Which four of a token's results a lane has: neighbours where a row's length lets four
// be one aligned word, else two pairs or four values, each with those of the other
// lanes beside it.
struct FourOf {
    int run;      // results of one word
    int at[4];    // from the tile's first row on
    int inside;   // a bit for each of them inside the matrix
    template <int kLanes>
    static __device__ __forceinline__ FourOf of(int l, int rows, int n0) {
        FourOf f;
        f.run = (rows & 3) == 0 ? 4 : (rows & 1) == 0 ? 2 : 1;  // (n0 is a multiple of four)
        f.inside = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f.at[e] = f.run == 4 ? 4 * l + e : f.run == 2 ? 2 * l + (e & 1) + 2 * kLanes * (e >> 1) : l + kLanes * e;
            f.inside |= (n0 + f.at[e] < rows) << e;
        }
        return f;
    }
    // from shared memory (all of a tile's sums are there)
    __device__ __forceinline__ float4 sums(const float* row) const {
        if (run == 4) return *reinterpret_cast<const float4*>(row + at[0]);
        return make_float4(row[at[0]], row[at[1]], row[at[2]], row[at[3]]);
    }
    // from a token's row, first value of the tile on
    template <typename T>
    __device__ __forceinline__ float4 load(const T* row) const {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (run == 4) {
            if ((inside & 1) == 0) return v;
            if constexpr (sizeof(T) == 4) return __ldg(reinterpret_cast<const float4*>(row + at[0]));
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(row + at[0]));
            return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                               __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
        }
        if (inside & 1) v.x = to_float(row[at[0]]);
        if (inside & 2) v.y = to_float(row[at[1]]);
        if (inside & 4) v.z = to_float(row[at[2]]);
        if (inside & 8) v.w = to_float(row[at[3]]);
        return v;
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, float4 v) const {
        if (run == 4) {
            if ((inside & 1) == 0) return;
            if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(row + at[0]) = v;
            else *reinterpret_cast<uint2*>(row + at[0]) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        } else if (run == 2) {
            if constexpr (sizeof(T) == 4) {
                if (inside & 1) *reinterpret_cast<float2*>(row + at[0]) = make_float2(v.x, v.y);
                if (inside & 4) *reinterpret_cast<float2*>(row + at[2]) = make_float2(v.z, v.w);
            } else {
                if (inside & 1) *reinterpret_cast<uint32_t*>(row + at[0]) = pack_bf16(v.x, v.y);
                if (inside & 4) *reinterpret_cast<uint32_t*>(row + at[2]) = pack_bf16(v.z, v.w);
            }
        } else {
            if (inside & 1) row[at[0]] = from_float<T>(v.x);
            if (inside & 2) row[at[1]] = from_float<T>(v.y);
            if (inside & 4) row[at[2]] = from_float<T>(v.z);
            if (inside & 8) row[at[3]] = from_float<T>(v.w);
        }
    }
};

// The same for one matrix: z = sum + bias, y = act(z) + residual.  A warp takes a token's
// 128 rows, four a lane, of four tokens at a time, so that their residuals are on their
// way together.  (In pairs as above the four warps' instructions bounded short products:
// 64 experts of 64 tokens, 7168 x 2048, 343 us against 294.)
template <typename T>
__device__ __forceinline__ void emit_linear(const TcArgs& p, const float* sums, int n0, int rows, int m0,
                                            int count, int expert, const Team& team) {
    constexpr int kAtOnce = 4;
    const int warps = team.threads >> 5;
    const FourOf four = FourOf::of<32>(team.thread & 31, rows, n0);
    float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.bias != nullptr) bias = four.load(p.bias + static_cast<size_t>(expert) * rows + n0);
    for (int c0 = team.thread >> 5; c0 < count; c0 += kAtOnce * warps) {
        float4 v[kAtOnce], r[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int c = min(c0 + u * warps, count - 1);
            v[u] = four.sums(sums + c * kSumPitch);
            r[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.residual != nullptr)
                r[u] = four.load(static_cast<const T*>(p.residual) + static_cast<size_t>(m0 + c) * rows + n0);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int c = c0 + u * warps;
            if (c >= count) break;
            const size_t to = static_cast<size_t>(m0 + c) * rows + n0;
            float4 o = make_float4(v[u].x + bias.x, v[u].y + bias.y, v[u].z + bias.z, v[u].w + bias.w);
            if (p.z != nullptr) four.store(static_cast<T*>(p.z) + to, o);
            if (p.act != kActNone) {
                o.x = act_value<sizeof(T) == 2>(o.x, p.act);
                o.y = act_value<sizeof(T) == 2>(o.y, p.act);
                o.z = act_value<sizeof(T) == 2>(o.z, p.act);
                o.w = act_value<sizeof(T) == 2>(o.w, p.act);
            }
            four.store(static_cast<T*>(p.y) + to,
                       make_float4(o.x + r[u].x, o.y + r[u].y, o.z + r[u].z, o.w + r[u].w));
        }
    }
}

template <int kX, bool kTma, Tc kMode, typename T, bool kSeg>
__global__ void __launch_bounds__(kThreads, 1)
ffn_tc_kernel(TcArgs p, const __grid_constant__ TcMaps maps) {
    using C = Cfg<kX, kTma, kMode>;
    constexpr bool kBack = kMode == Tc::kBackward;
    constexpr bool kDuo = C::kDuo;
    constexpr int S = C::kStages;
    constexpr int kSplit0 = kMode == Tc::kGated ? kRows / 2 : kRows;  // tile rows of w0
    constexpr bool kTwo = kMode == Tc::kGated || kBack;  // (backward of one matrix: w1 is w0)
    extern __shared__ uint8_t smem_dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rows = kBack ? p.K : p.N;  // rows of the product
    const int peer = kDuo ? static_cast<int>(blockIdx.x & 1) : 0;
    Work work;
    work.parts = p.parts;
    work.part = blockIdx.x / C::kCtas % p.parts;
    work.w = blockIdx.x / (C::kCtas * p.parts);
    work.workers = gridDim.x / (C::kCtas * p.parts);
    work.quads = p.quads;
    work.tiles = p.tiles;
    work.whole = p.whole;
    if (kSeg) {
        // (the plan counts what there could be; all are whole)
        pdl_wait_prerequisites();
        work.tiles = work.whole = *p.table_count * p.row_units;
    }
    Segment sg;
    // first row (backward: column k) of a tile, first token and how many, its MMA N,
    // and whose matrices
    auto row0 = [&](int tile) { return (C::kCtas * (tile % p.row_units) + peer) * kSplit0; };
    auto token0 = [&](int tile) {
        return kSeg ? p.table[tile / p.row_units].y : tile / p.row_units * kX;
    };
    auto tokens_of = [&](int tile) {
        return kSeg ? p.table[tile / p.row_units].z : min(kX, p.M - tile / p.row_units * kX);
    };
    auto expert_of = [&](int tile) { return kSeg ? p.table[tile / p.row_units].x : 0; };
    auto mma_n = [&](int tile) {
        const int tokens = tokens_of(tile);
        return kDuo ? (tokens + 31) & ~31 : (tokens + 15) & ~15;
    };

    const uint32_t bar_xfull = sbase + C::kOffBar;
    const uint32_t bar_afull = bar_xfull + 8 * S;
    const uint32_t bar_peer = bar_afull + 8 * S;  // (of the first CTA)
    const uint32_t bar_empty = bar_peer + 8 * S;
    const uint32_t bar_raw = bar_empty + 8 * S;
    const uint32_t bar_rawempty = bar_raw + 8 * C::kRaw;
    const uint32_t bar_accfull = bar_rawempty + 8 * C::kRaw;
    const uint32_t bar_accempty = bar_accfull + 16;  // (of the first CTA)
    const uint32_t bar_drain = bar_accempty + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    volatile int* shared_word = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
    unsigned int* err = &g_tc_error;

    if (warp == 0) {
        for (int s = lane; s < S; s += 32) {
            mbar_init(bar_xfull + 8 * s, 1);               // the producer's expect-tx arrival
            mbar_init(bar_afull + 8 * s, C::kGroupWarps);  // the warps of its group
            mbar_init(bar_peer + 8 * s, 1);                // the second CTA's waiter
            mbar_init(bar_empty + 8 * s, 1);  // MMA commits
        }
        for (int r = lane; r < C::kRaw; r += 32) {
            mbar_init(bar_raw + 8 * r, kTma || !kBack ? 1 : kDecWarps);
            mbar_init(bar_rawempty + 8 * r, kBack ? C::kGroupWarps : kDecWarps);
        }
        if (lane < 2) {
            mbar_init(bar_accfull + 8 * lane, 1);
            mbar_init(bar_accempty + 8 * lane, 4 * C::kCtas);  // epilogue warps
        }
        if (lane == 0) {
            mbar_init(bar_drain, 1);
            *abort_flag = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc<kDuo>(smem_u32(tmem_slot), C::kTmemCols);
    fence_before();
    if (kDuo) cluster_sync();  // the other CTA's barriers are set up
    else __syncthreads();
    fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
    const uint32_t raw0 = sbase + C::kOffRaw;
    auto hand_over = [&]() {  // the waiter and the issuer
        asm volatile("bar.sync 1, 64;" ::: "memory");
    };

    if (warp < kDecWarps) {
        // ---------------- weight decoders ----------------
        const int td = threadIdx.x;
        if (!kTma && kBack && !p.const_weights) pdl_wait_prerequisites();
        // Raw rows 112 bytes apart fall on eight banks: every other eight lanes take
        // the halves of a segment's 16 bytes in the other order, and store them
        // accordingly (where the store has an address of the lane's own).
        const int turn = kTma && !C::kTmemA ? (lane >> 3) & 1 : 0;
        // wait for stage i's place, counted over all segments
        auto stage_free = [&](int i) -> bool {
            return i < S || __all_sync(0xFFFFFFFFu,
                                       mbar_wait_bounded(bar_empty + 8 * (i % S), ((i / S) - 1) & 1,
                                                         abort_flag, err, kErrTimeoutEmpty));
        };
        auto publish = [&](int i) {
            fence_async_smem();  // this thread's stores -> visible to the MMA
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_afull + 8 * (i % S));
        };
        // This warp is done with a raw slot.  Its words are read in the generic proxy
        // and overwritten in the async proxy (the next block's copy), so each lane
        // orders its reads before the copy by a proxy fence: the barrier alone does
        // not, and without it loads still on their way were seen to bring the next
        // block's bytes.
        [[maybe_unused]] auto raw_read = [&](uint32_t bar) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        if constexpr (kBack) {
            // group (four warps) takes every fourth stage: warp = 32 weight rows
            // and a segment, lane = the row, all four shifts
            const int own = warp >> 2, tg = td & 127;
            const int seg = warp & 1, n = 32 * ((warp >> 1) & 1) + lane;
            bool ok = true;  // a warp that gave up still passes the group's barriers
            int i = own;     // this group's stages, counted over all segments
            // without TMA: the next stage to fetch (a slot ahead of the decode)
            Segment fetch = {};
            int fetch_index = 0, fetch_q = 0, fetched = own;
            bool more = false;
            [[maybe_unused]] auto fetch_next = [&]() {
                if (more) {
                    issue_raw_rows(p, raw0 + (fetched % C::kRaw) * C::kRawBytes, 4 * fetch_q + own,
                                   expert_of(fetch.tile), row0(fetch.tile) / kQK,
                                   (row0(fetch.tile) / kRows) & 1, tg);
                    fetched += 4;
                    if (++fetch_q == fetch.q1) {
                        more = work.segment(++fetch_index, fetch);
                        fetch_q = fetch.q0;
                    }
                } else {
                    cp_async_commit();
                }
            };
            if constexpr (!kTma) {
                more = work.segment(0, fetch);
                fetch_q = fetch.q0;
                fetch_next();
            }
            for (int index = 0; work.segment(index, sg); ++index) {
                const int block = row0(sg.tile) / kQK, half = (row0(sg.tile) / kRows) & 1;
                for (int q = sg.q0; q < sg.q1; ++q, i += 4) {
                    const int slot = i % C::kRaw;
                    const uint32_t raw = raw0 + slot * C::kRawBytes + n * C::kRawPitch;
                    uint32_t at_sc = raw, at_q = raw + 8, at_d = raw + 40;
                    if constexpr (kTma) {
                        ok = ok && __all_sync(0xFFFFFFFFu,
                                              mbar_wait_bounded(bar_raw + 8 * slot, (i / C::kRaw) & 1,
                                                                abort_flag, err, kErrTimeoutEmpty));
                        const uint32_t at = raw + ((kBlockBytes * block) & 15);  // (a 16-byte boundary)
                        at_sc = at + 8 * half;
                        at_q = at + 16 + 32 * half;
                        at_d = at + 80;
                    } else {
                        // the group's other slot was read before this barrier
                        asm volatile("bar.sync %0, 128;" ::"r"(3 + own) : "memory");
                        fetch_next();
                        cp_async_wait<1>();
                        asm volatile("bar.sync %0, 128;" ::"r"(3 + own) : "memory");
                    }
                    if (!ok) continue;
                    uint32_t qw[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        qw[e] = ld_shared_u32(at_q + 16 * seg + 4 * (e & 1) + 8 * ((e >> 1) ^ turn));
                    const uint32_t sc0 = ld_shared_u32(at_sc) >> (8 * seg);
                    const uint32_t sc1 = ld_shared_u32(at_sc + 4) >> (8 * seg);
                    const uint32_t dd = ld_shared_u32(at_d);
                    const float d = f16_bits_to_float(dd), dmin = f16_bits_to_float(dd >> 16);
                    uint32_t o[4][8];
                    decode_segment<0>(qw, sc0 & 0xFFu, d, dmin, o[0]);
                    decode_segment<1>(qw, (sc0 >> 16) & 0xFFu, d, dmin, o[1]);
                    decode_segment<2>(qw, sc1 & 0xFFu, d, dmin, o[2]);
                    decode_segment<3>(qw, (sc1 >> 16) & 0xFFu, d, dmin, o[3]);
                    if constexpr (kTma) raw_read(bar_rawempty + 8 * slot);
                    ok = stage_free(i);
                    if (!ok) continue;
                    // row n of the stage: 128 bytes of columns 64 c .. at 8192 c +
                    // 128 n, its 16-byte chunks swizzled by n % 8
                    const uint32_t dst = sbase + C::kOffA + (i % S) * kABytes + 128 * n;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            st_shared_v4(dst + 8192 * (j >> 1) +
                                             (((4 * (j & 1) + 2 * seg + c) ^ (n & 7) ^ turn) << 4),
                                         o[j][4 * c], o[j][4 * c + 1], o[j][4 * c + 2], o[j][4 * c + 3]);
                    publish(i);
                }
            }
        } else {
            // group (four warps) takes stage `own` of every block, thread = a
            // weight row: shifts 2 (own % 2) and + 1 of half own / 2, both segments
            const int row = 32 * (warp & 3) + lane, own = warp >> 2;
            bool ok = true;
            int b = 0;  // blocks, counted over all segments
            for (int index = 0; ok && work.segment(index, sg); ++index) {
                // (without maps of single rows: the row's place in a slot, and where
                // in its group it starts, -1 if it comes by the word)
                [[maybe_unused]] int place = row, row_at = 0;
                if constexpr (!kTma) {
                    const bool word = row0(sg.tile) + row % kSplit0 >= 4 * p.groups;
                    place = raw_place<kSplit0>(row, word && p.groups > 0);
                    row_at = word ? -1 : (row & 3) * (p.K / kQK) * kBlockBytes;
                }
                for (int q = sg.q0; q < sg.q1 && ok; ++q, ++b) {
                    const int buf = b % C::kRaw;
                    uint32_t mine = raw0 + buf * C::kRawBytes + place * C::kRawPitch;
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar_raw + 8 * buf, (b / C::kRaw) & 1,
                                                                   abort_flag, err, kErrTimeoutEmpty));
                    if (!ok) break;
                    // (what was copied starts at a 16-byte boundary)
                    mine += kTma ? 4 * (q & 3) : row_at < 0 ? 0 : (row_at + kBlockBytes * q) & 15;
                    const int half = own >> 1;
                    const uint32_t sc = ld_shared_u32(mine + 8 * half + 4 * (own & 1));
                    uint32_t qw[2][4];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        qw[e >> 2][e & 3] = ld_shared_u32(mine + 16 + 32 * half + 16 * (e >> 2) + 4 * (e & 1) +
                                                          8 * (((e >> 1) & 1) ^ turn));
                    const uint32_t dd = ld_shared_u32(mine + 80);
                    const float d = f16_bits_to_float(dd), dmin = f16_bits_to_float(dd >> 16);
                    uint32_t o[4][8];  // (shift, segment)
                    if (own & 1) {
                        decode_segment<2>(qw[0], sc & 0xFFu, d, dmin, o[0]);
                        decode_segment<2>(qw[1], (sc >> 8) & 0xFFu, d, dmin, o[1]);
                        decode_segment<3>(qw[0], (sc >> 16) & 0xFFu, d, dmin, o[2]);
                        decode_segment<3>(qw[1], sc >> 24, d, dmin, o[3]);
                    } else {
                        decode_segment<0>(qw[0], sc & 0xFFu, d, dmin, o[0]);
                        decode_segment<0>(qw[1], (sc >> 8) & 0xFFu, d, dmin, o[1]);
                        decode_segment<1>(qw[0], (sc >> 16) & 0xFFu, d, dmin, o[2]);
                        decode_segment<1>(qw[1], sc >> 24, d, dmin, o[3]);
                    }
                    raw_read(bar_rawempty + 8 * buf);
                    const int i = 4 * b + own;
                    ok = stage_free(i);
                    if (!ok) break;
                    if constexpr (C::kTmemA) {
                        fence_after();  // the MMAs that read this stage are done
                        const uint32_t col = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) +
                                             C::kColA + 32u * (i % S);
#pragma unroll
                        for (int j = 0; j < 4; ++j) tmem_store8(col + 8u * j, o[j]);
                        tmem_store_wait();
                        fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar_afull + 8 * (i % S));
                    } else {
                        const uint32_t dst = sbase + C::kOffA + (i % S) * kABytes;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                st_shared_v4(dst + 128 * row + (((2 * j + c) ^ (row & 7) ^ turn) << 4), o[j][4 * c],
                                             o[j][4 * c + 1], o[j][4 * c + 2], o[j][4 * c + 3]);
                        publish(i);
                    }
                }
            }
        }
        if constexpr (!kTma && kBack) asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == kMmaWarp && peer == 0) {
        // ---------------- MMA issuer ----------------
        // It meets the waiter at named barrier 1 once for every two stages, when
        // both are filled and, at a tile's first, its set of sums is free; both
        // pass it the same number of times, whatever happens.  Nothing but MMAs
        // and commits stands between its MMAs.  The thread comes from
        // elect.sync, not from a test of its lane: only so are an MMA's
        // descriptors computed in uniform registers, without a transfer each
        // before every MMA (512 tokens, 14336 x 4096: 82 us against 93).
        const uint64_t xdesc0 = sw128_desc(sbase);
        const uint64_t adesc0 = kBack ? sw128_mn_desc(sbase + C::kOffA, 8192)
                                      : sw128_desc(sbase + C::kOffA);
        int i0 = 0;  // stages, counted over all segments
        for (int index = 0; work.segment(index, sg); ++index) {
            const uint32_t idesc = bf16_idesc(C::kCtas * kRows, mma_n(sg.tile)) | (kBack ? kIdescAMnMajor : 0u);
            const uint32_t acc = tmem + (index & 1) * C::kAccCols;
            const int n_iters = 4 * (sg.q1 - sg.q0);
            for (int l0 = 0; l0 < n_iters; l0 += C::kHand, i0 += C::kHand) {
                hand_over();
                if (elect_one() && !*abort_flag) {
                    fence_after();
#pragma unroll
                    for (int u = 0; u < C::kHand; ++u) {
                        const int s = (i0 + u) % S;
                        const uint64_t xdesc = xdesc0 + static_cast<uint64_t>(s * (C::kXStage >> 4));
                        const uint64_t adesc = adesc0 + static_cast<uint64_t>(s * (kABytes >> 4));
#pragma unroll
                        for (int kk = 0; kk < kStageK / 16; ++kk) {
                            const uint32_t add = l0 + u > 0 || kk > 0;
                            if constexpr (C::kTmemA)
                                mma_tmem_a(acc, tmem + C::kColA + 32u * s + 8u * kk, xdesc + 2u * kk,
                                           idesc, add);
                            else  // (backward: a K-step is 16 rows)
                                mma<kDuo>(acc, adesc + (kBack ? 128u : 2u) * kk, xdesc + 2u * kk, idesc, add);
                        }
                        commit<kDuo>(bar_empty + 8 * s);
                    }
                    if (l0 + C::kHand == n_iters) commit<kDuo>(bar_accfull + 8 * (index & 1));
                }
                __syncwarp();
            }
        }
        if (elect_one() && *abort_flag) {
            // no MMA may still write TMEM when it is freed
            commit<kDuo>(bar_drain);
            volatile int no_abort = 0;
            mbar_wait_bounded(bar_drain, 0, &no_abort, err, kErrTimeoutDrain);
        }
        __syncwarp();
    } else if (warp == kWaitWarp) {
        // ---------------- stage waiter ----------------
        // Two CTAs: the second one's waiter reports each of its stages to the
        // first's, which waits for both.
        int i0 = 0;
        for (int index = 0; work.segment(index, sg); ++index) {
            const int n_iters = 4 * (sg.q1 - sg.q0);
            for (int l0 = 0; l0 < n_iters; l0 += C::kHand, i0 += C::kHand) {
                if (lane == 0 && !*abort_flag) {
                    bool ok = peer == 1 || l0 > 0 || index < 2 ||
                              wait_peer_bounded(bar_accempty + 8 * (index & 1), ((index >> 1) - 1) & 1,
                                                abort_flag, err, kErrTimeoutAccum);
#pragma unroll
                    for (int u = 0; u < C::kHand; ++u) {
                        const int i = i0 + u;
                        const uint32_t at = 8 * (i % S), phase = (i / S) & 1;
                        ok = ok && mbar_wait_bounded(bar_xfull + at, phase, abort_flag, err, kErrTimeoutFull) &&
                             mbar_wait_bounded(bar_afull + at, phase, abort_flag, err, kErrTimeoutFull);
                        if (kDuo && ok && peer == 1) arrive_first_of_pair(bar_peer + at);
                        if (kDuo && peer == 0)
                            ok = ok && wait_peer_bounded(bar_peer + at, phase, abort_flag, err, kErrTimeoutFull);
                    }
                }
                __syncwarp();
                if (peer == 0) hand_over();
            }
        }
    } else if (warp == kWWarp) {
        // ---------------- raw weight blocks ----------------
        if (kTma && lane == 0) {
            tma_prefetch_map(&maps.w0);
            if (kTwo) tma_prefetch_map(&maps.w1);
            if (!p.const_weights) pdl_wait_prerequisites();
            int b = 0;
            bool ok = true;
            for (int index = 0; ok && work.segment(index, sg); ++index) {
                const int n0 = row0(sg.tile), expert = expert_of(sg.tile);
                for (int r = 0; ok && r < (sg.q1 - sg.q0) * (kBack ? 4 : 1); ++r, ++b) {
                    const int buf = b % C::kRaw;
                    ok = b < C::kRaw ||
                         mbar_wait_bounded(bar_rawempty + 8 * buf, ((b / C::kRaw) - 1) & 1, abort_flag,
                                           err, kErrTimeoutEmpty);
                    if (!ok) break;
                    const uint32_t dst = sbase + C::kOffRaw + buf * C::kRawBytes;
                    const uint32_t bar = bar_raw + 8 * buf;
                    mbar_arrive_expect_tx(bar, C::kRawBytes);
                    if constexpr (kBack) {
                        const int stage = 4 * sg.q0 + r;
                        const bool up = stage >= p.half_stages;
                        load_weights<kSeg>(dst, up ? &maps.w1 : &maps.w0, (kBlockBytes * (n0 / kQK)) & ~15,
                                           kStageK * (up ? stage - p.half_stages : stage), expert, bar);
                    } else {
                        const int x = (kBlockBytes * (sg.q0 + r)) & ~15;
                        load_weights<kSeg>(dst, &maps.w0, x, n0, expert, bar);
                        if (kMode == Tc::kGated)
                            load_weights<kSeg>(dst + kSplit0 * kBoxBytes, &maps.w1, x, n0, expert, bar);
                    }
                }
            }
            if (*abort_flag) linger();
        }
        if constexpr (!kTma && !kBack) {
            // Rows that do not all start at 16 bytes: every fourth row does, so a map
            // of groups of four rows serves each row of the group by a copy of its
            // own, and the matrix's last rows (or all, off 16 bytes) come by the
            // word.  (The decoders' own 4-byte copies kept them in step: 4999 x 2816,
            // 77 tokens, 22.4 us; a bulk copy for each row's block 42.)
            if (lane == 0 && p.groups > 0) {
                tma_prefetch_map(&maps.w0);
                if (kTwo) tma_prefetch_map(&maps.w1);
            }
            if (!p.const_weights) pdl_wait_prerequisites();
            const size_t row_bytes = static_cast<size_t>(p.K / kQK) * kBlockBytes;
            int b = 0;
            bool ok = true;
            for (int index = 0; ok && work.segment(index, sg); ++index) {
                const int n0 = row0(sg.tile), expert = expert_of(sg.tile);
                const size_t matrix = static_cast<size_t>(expert) * p.N * row_bytes;
                const bool words = n0 + kSplit0 > 4 * p.groups;
                for (int q = sg.q0; ok && q < sg.q1; ++q, ++b) {
                    const int buf = b % C::kRaw;
                    ok = b < C::kRaw ||
                         __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar_rawempty + 8 * buf,
                                                                   ((b / C::kRaw) - 1) & 1, abort_flag, err,
                                                                   kErrTimeoutEmpty));
                    if (!ok) break;
                    const uint32_t bar = bar_raw + 8 * buf, slot = raw0 + buf * C::kRawBytes;
                    if (words) {
                        for (int r = lane; r < kRows; r += 32) {
                            const int n = n0 + r % kSplit0;
                            if (n < 4 * p.groups || n >= p.N) continue;
                            const uint32_t* src = reinterpret_cast<const uint32_t*>(
                                (r < kSplit0 ? p.w0 : p.w1) + matrix + n * row_bytes +
                                static_cast<size_t>(kBlockBytes) * q);
                            const uint32_t dst = slot + raw_place<kSplit0>(r, p.groups > 0) * C::kRawPitch;
                            uint32_t v[kWordsPerBlock];
#pragma unroll
                            for (int w = 0; w < kWordsPerBlock; ++w) v[w] = __ldg(src + w);
#pragma unroll
                            for (int w = 0; w < kWordsPerBlock; ++w)
                                asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + 4 * w), "r"(v[w]) : "memory");
                        }
                        __syncwarp();
                    }
                    if (lane == 0 && p.groups == 0) mbar_arrive(bar);
                    if (lane == 0 && p.groups > 0) {
                        mbar_arrive_expect_tx(bar, kRows * kBoxBytes);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int x = static_cast<int>((j * row_bytes + kBlockBytes * q) & ~size_t(15));
                            load_weights<kSeg>(slot + j * (kSplit0 / 4) * kBoxBytes, &maps.w0, x, n0 / 4, expert, bar);
                            if (kMode == Tc::kGated)
                                load_weights<kSeg>(slot + (kSplit0 + j * (kSplit0 / 4)) * kBoxBytes, &maps.w1, x,
                                            n0 / 4, expert, bar);
                        }
                    }
                }
            }
            if (*abort_flag) linger();
        }
        __syncwarp();
    } else if (warp == kXWarp) {
        // ---------------- token stages ----------------
        if (lane == 0) {
            if (p.xa == nullptr) {
                tma_prefetch_map(&maps.x0);
                if (kBack) tma_prefetch_map(&maps.x1);
            }
            if (!p.tokens_ready) {
                pdl_wait_prerequisites();  // the tokens
                pdl_allow_dependents();
            }
            int i = 0;
            bool ok = true;
            for (int index = 0; ok && work.segment(index, sg); ++index) {
                // two CTAs: this one holds tokens [peer N / 2, peer N / 2 + N / 2)
                const int held = mma_n(sg.tile) / C::kCtas;
                const int m_held = token0(sg.tile) + peer * held;
                const uint8_t* src = p.xa +
                                     static_cast<size_t>(m_held / kSuperRows) * 4 * p.quads * kSuperBytes +
                                     static_cast<size_t>(m_held % kSuperRows) * (kStageK * 2);
                const uint32_t bytes = p.xa != nullptr ? held * (kStageK * 2) : C::kXStage;
                for (int stage = 4 * sg.q0; stage < 4 * sg.q1; ++stage, ++i) {
                    ok = i < S || mbar_wait_bounded(bar_empty + 8 * (i % S), ((i / S) - 1) & 1, abort_flag,
                                                    err, kErrTimeoutEmpty);
                    if (!ok) break;
                    const uint32_t dst = sbase + (i % S) * C::kXStage, bar = bar_xfull + 8 * (i % S);
                    mbar_arrive_expect_tx(bar, bytes);
                    if (p.xa != nullptr) {
                        bulk_copy_g2s(dst, src + static_cast<size_t>(stage) * kSuperBytes, bytes, bar);
                    } else {
                        // (tokens past M and, backward, weight rows past N read as zeros)
                        const bool up = kBack && stage >= p.half_stages;
                        tma_load_2d(dst, up ? &maps.x1 : &maps.x0,
                                    kStageK * (up ? stage - p.half_stages : stage), m_held, bar);
                    }
                }
            }
            if (*abort_flag) linger();
        }
        __syncwarp();
    }
    // Results of `count` tokens (from m on) of a tile from their sums; the last
    // tile's (`final`) lie where the rings were, from token slot `slot` on.
    auto bring_out = [&](float* base, bool final, int n0, [[maybe_unused]] int expert, int m, int count,
                         const Team& team, int slot = 0, int slot0 = 0) {
        if constexpr (kMode == Tc::kLora) {
            uint32_t* tbuf = reinterpret_cast<uint32_t*>(final ? base + kX * kSumPitch
                                                               : reinterpret_cast<float*>(smem + C::kOffT));
            const int* id_buf = reinterpret_cast<const int*>(smem + C::kOffIds);
            // (base holds the sums of the tile's tokens from slot0 on)
            add_adapters(base - slot0 * kSumPitch, tbuf, id_buf + slot0 + slot, id_buf + kX + slot0 + slot,
                         p, n0, m - slot0, count, team);
        }
        if constexpr (kMode == Tc::kLinear)
            emit_linear<T>(p, base + slot * kSumPitch, n0, rows, m + slot, count, expert, team);
        else
            emit<kMode, T>(p, base + slot * kSumPitch, n0, rows, m + slot, count, team);
    };
    const bool brings_out = warp < kDecWarps || warp >= kEpiWarp0;
    if (brings_out) {
        // ---------------- epilogue: sums -> results ----------------
        // (what is written here, and t, may still be in use by the grid before)
        pdl_wait_prerequisites();
        if (p.tokens_ready) pdl_allow_dependents();
        const int segments = work.count();
        // the decoders come for the last segment
        for (int index = warp < kDecWarps ? (kSeg ? max(segments - 1, 0) : segments - 1) : 0;
             work.segment(index, sg); ++index) {
            const bool final = index == segments - 1;
            Team team;
            team.thread = warp < kDecWarps ? static_cast<int>(threadIdx.x) + 128
                                           : static_cast<int>(threadIdx.x) - 32 * kEpiWarp0;
            team.threads = final ? 128 + kDecThreads : 128;
            team.barrier = final ? 7 : 2;
            if constexpr (kMode == Tc::kLora) {
                if (warp >= kEpiWarp0) {
                    const int m0 = token0(sg.tile), tokens = min(kX, p.M - m0);
                    int* id_buf = reinterpret_cast<int*>(smem + C::kOffIds);
                    // (of parts of K, each has a share of the tokens)
                    const int groups = (tokens + 7) / 8;
                    sort_tokens<kX>(id_buf, id_buf + kX, p, m0, tokens, 8 * (work.part * groups / p.parts),
                                    8 * ((work.part + 1) * groups / p.parts), final ? kX : kChunk, team.thread);
                }
            }
            mbar_wait_backoff(bar_accfull + 8 * (index & 1), (index >> 1) & 1, abort_flag, err,
                              kErrTimeoutAccum, 512);
            // all of the team go on, or none (after a time-out they still meet
            // the decoders at the last segment)
            team.sync();
            if (team.thread == 0) *shared_word = *abort_flag;
            team.sync();
            const bool stop = *shared_word != 0;
            team.sync();
            if (stop) continue;
            fence_after();
            // the last tile's sums take the place of the rings
            float* sums = reinterpret_cast<float*>(smem + (final ? 0 : C::kOffSums));
            const int chunk = final ? kX : kChunk;
            const int n0 = row0(sg.tile), m0 = token0(sg.tile), expert = expert_of(sg.tile);
            const int tokens = tokens_of(sg.tile);
            const int quarter = (team.thread >> 5) & 3, my_row = 32 * quarter + lane;
            const int strip = 16 * (team.thread >> 7), strips = 16 * (team.threads >> 7);
            const uint32_t t_lane = tmem + (index & 1) * C::kAccCols +
                                    (static_cast<uint32_t>(32 * quarter) << 16);
            // 16 tokens of this lane's row, from c0 on
            auto load_sums = [&](int c0, float (&v)[16]) { tmem_load16(t_lane + c0, v); };
            auto release = [&]() {  // the sums are read: their set may be reused
                if (final) return;  // (by none)
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kDuo) arrive_first_of_pair(bar_accempty + 8 * (index & 1));
                    else mbar_arrive(bar_accempty + 8 * (index & 1));
                }
            };
            int first = 0, last = 0;
            if (sg.run >= 0) {
                // A run of a cut tile: its sums go to the workspace, and the CTA
                // that counts last adds the runs.  The barrier and the fence
                // order every thread's stores before the count; the second fence
                // orders the count before the loads.
                float* mine = p.partial + static_cast<size_t>((2 * work.w + sg.run) * C::kCtas + peer) * (kX * kRows);
                for (int c0 = strip; c0 < tokens; c0 += strips) {
                    float v[16];
                    load_sums(c0, v);
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        if (c0 + q < tokens) mine[(c0 + q) * kRows + my_row] = v[q];
                }
                release();
                work.sharers(sg.tile, first, last);
                team.sync();
                if (team.thread == 0) {
                    __threadfence();
                    const unsigned before =
                        atomicAdd(p.counts + (sg.tile - p.whole) * C::kCtas + peer, 1u);
                    __threadfence();
                    *shared_word = before == static_cast<unsigned>(last - first);
                }
                team.sync();
                const bool add = *shared_word != 0;
                team.sync();  // (the word is read before the next segment writes it)
                if (!add) continue;
            }
            for (int c0 = 0; c0 < tokens && !(final && p.parts > 1); c0 += chunk) {
                const int count = min(chunk, tokens - c0);
                if (sg.run < 0) {
                    for (int h = strip; h < count; h += strips) {
                        float v[16];
                        load_sums(c0 + h, v);
#pragma unroll
                        for (int q = 0; q < 16; ++q) sums[(h + q) * kSumPitch + my_row] = v[q];
                    }
                    if (c0 + chunk >= tokens) release();
                } else {
                    // two float4 of up to three runs at a time: latency bounds it
                    const int quads = count * (kRows / 4);
                    auto run_sums = [&](int v) {
                        return reinterpret_cast<const float4*>(
                                   p.partial + static_cast<size_t>((2 * v + work.run_of(v, sg.tile)) * C::kCtas + peer) *
                                                   (kX * kRows)) + c0 * (kRows / 4);
                    };
                    for (int i0 = team.thread; i0 < quads; i0 += 2 * team.threads) {
                        const int i1 = i0 + team.threads;
                        float4 a[2];
                        a[0] = a[1] = make_float4(0.f, 0.f, 0.f, 0.f);
                        for (int v = first; v <= last; v += 3) {
                            float4 x[3][2];
#pragma unroll
                            for (int z = 0; z < 3; ++z) {
                                x[z][0] = x[z][1] = make_float4(0.f, 0.f, 0.f, 0.f);
                                if (v + z > last) continue;
                                const float4* src = run_sums(v + z);
                                x[z][0] = __ldcg(src + i0);
                                if (i1 < quads) x[z][1] = __ldcg(src + i1);
                            }
#pragma unroll
                            for (int z = 0; z < 3; ++z)
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    a[u].x += x[z][u].x;
                                    a[u].y += x[z][u].y;
                                    a[u].z += x[z][u].z;
                                    a[u].w += x[z][u].w;
                                }
                        }
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int i = u ? i1 : i0;
                            if (i < quads)
                                *reinterpret_cast<float4*>(sums + (i / (kRows / 4)) * kSumPitch +
                                                           4 * (i % (kRows / 4))) = a[u];
                        }
                    }
                }
                team.sync();
                bring_out(sums, final, n0, expert, m0 + c0, count, team, 0, c0);
                team.sync();
            }
            if (final && p.parts > 1 && sg.run < 0) {
                // parts of K: the sums wait here for the cluster
                for (int h = strip; h < tokens; h += strips) {
                    float v[16];
                    load_sums(h, v);
#pragma unroll
                    for (int q = 0; q < 16; ++q) sums[(h + q) * kSumPitch + my_row] = v[q];
                }
            }
        }
    }
    if (p.parts > 1) {
        // Every thread of the cluster passes its barriers, whatever happened
        // before.  Part z adds its share of the tokens (whole groups of eight)
        // over the parts in order and brings them out; the barrier at the end
        // keeps every part's sums alive until all are read.
        fence_before();
        __syncwarp();
        cluster_sync();
        const bool any = work.segment(0, sg);
        if (brings_out && (any || !kSeg)) {
            Team team;
            team.thread = warp < kDecWarps ? static_cast<int>(threadIdx.x) + 128
                                           : static_cast<int>(threadIdx.x) - 32 * kEpiWarp0;
            team.threads = 128 + kDecThreads;
            team.barrier = 7;
            const int n0 = row0(sg.tile), m0 = token0(sg.tile), expert = expert_of(sg.tile);
            const int tokens = tokens_of(sg.tile), groups = (tokens + 7) / 8;
            const int first = 8 * (work.part * groups / p.parts);
            const int count = min(tokens, 8 * ((work.part + 1) * groups / p.parts)) - first;
            float* sums = reinterpret_cast<float*>(smem) + first * kSumPitch;
            for (int j = team.thread; j < count * (kRows / 4); j += team.threads) {
                const int i = j / (kRows / 4) * (kSumPitch / 4) + j % (kRows / 4);
                const uint32_t at = smem_u32(sums) + 16 * i;
                float4 v[kMaxParts];
#pragma unroll
                for (int z = 0; z < kMaxParts; ++z)
                    if (z < p.parts) v[z] = load_cluster4(at, C::kCtas * z + peer);
                float4 a = v[0];
#pragma unroll
                for (int z = 1; z < kMaxParts; ++z)
                    if (z < p.parts) {
                        a.x += v[z].x;
                        a.y += v[z].y;
                        a.z += v[z].z;
                        a.w += v[z].w;
                    }
                reinterpret_cast<float4*>(sums)[i] = a;
            }
            team.sync();
            if (*abort_flag == 0 && count > 0)
                bring_out(reinterpret_cast<float*>(smem), true, n0, expert, m0, count, team, first);
        }
    }

    fence_before();
    __syncwarp();
    if (kDuo || p.parts > 1) cluster_sync();
    else __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        tmem_free<kDuo>(tmem, C::kTmemCols);
    }
}

// A bf16 [rows, cols] matrix with rows `pitch` apart, in boxes of box_rows x 64
// columns, 128-byte swizzled.
bool make_token_map(CUtensorMap* map, const void* x, int rows, int cols, int pitch, int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * 2};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kStageK), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t elem[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(x), dims, strides, box,
                  elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kX, bool kTma, Tc kMode, typename T, bool kSeg>
cudaError_t launch_tc_as(const TcArgs& a, const Plan& plan, const TcMaps& maps, int device,
                         cudaStream_t stream) {
    using C = Cfg<kX, kTma, kMode>;
    static std::atomic<bool> attr_done[64] = {};  // (set by any thread; setting twice does no harm)
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[device].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(ffn_tc_kernel<kX, kTma, kMode, T, kSeg>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   C::kSmemBytes);
        if (e != cudaSuccess) return e;
        attr_done[device].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(plan.workers * plan.ctas * plan.parts);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(plan.ctas * plan.parts);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = plan.ctas * plan.parts > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, ffn_tc_kernel<kX, kTma, kMode, T, kSeg>, a, maps);
}

}  // namespace

template <Tc kMode, typename T, bool kSeg>
cudaError_t launch_tc(TcArgs a, const Plan& plan, uint8_t* workspace, const void* x0, const void* x1,
                      int x_cols, int x_pitch, int device, cudaStream_t stream, int experts) {
    a.tiles = plan.tiles;
    a.row_units = plan.row_units;
    a.whole = plan.whole;
    a.parts = plan.parts;
    a.partial = reinterpret_cast<float*>(workspace);
    a.counts = reinterpret_cast<unsigned int*>(workspace + plan.partial);
    alignas(64) TcMaps maps;
    memset(&maps, 0, sizeof maps);
    constexpr bool kTwo = kMode == Tc::kGated || kMode == Tc::kBackward;
    const int rows = kTwo ? 64 : kRows;
    auto make_maps = [&](int group) {
        return make_weight_map(&maps.w0, a.w0, a.N, a.K, rows / group, group, kSeg ? experts : 0) &&
               (!kTwo || make_weight_map(&maps.w1, a.w1, a.N, a.K, rows / group, group, kSeg ? experts : 0));
    };
    const bool tma = make_maps(1);
    a.groups = !tma && kMode != Tc::kBackward && make_maps(4) ? a.N / 4 : 0;
    const int held = std::min(plan.x_rows, 128);  // tokens of a stage in one CTA
    if (a.xa == nullptr &&
        (!make_token_map(&maps.x0, x0, a.M, x_cols, x_pitch, held) ||
         (kMode == Tc::kBackward && !make_token_map(&maps.x1, x1, a.M, x_cols, x_pitch, held))))
        return cudaErrorNotSupported;
#define Q2K_TC_CASE(X)                                                              \
    case X:                                                                         \
        return tma ? launch_tc_as<X, true, kMode, T, kSeg>(a, plan, maps, device, stream) \
                   : launch_tc_as<X, false, kMode, T, kSeg>(a, plan, maps, device, stream);
    switch (plan.x_rows) {
        Q2K_TC_CASE(32)
        Q2K_TC_CASE(64)
        Q2K_TC_CASE(128)
        Q2K_TC_CASE(256)
    }
#undef Q2K_TC_CASE
    return cudaErrorInvalidValue;
}

}  // namespace q2k
