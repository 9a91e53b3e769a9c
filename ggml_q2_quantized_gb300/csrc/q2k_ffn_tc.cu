// Many tokens times Q2_K weights on the tensor cores (tcgen05): the gated
// feed-forward block, its backward product, and a projection with low-rank
// adapters.
//
// A CTA computes 128 rows of a product x up to 256 tokens: 16 warps decode Q2_K
// blocks into tensor memory (the MMA's A operand, one row of the product per
// lane), token stages of 64 K arrive by TMA in the 128-byte-swizzled layout that
// the MMA reads (the B operand; f32 tokens come from a bf16 image that a prepass
// writes in that layout), and f32 sums build up in tensor memory.
//
// Gated: the 128 rows are 64 rows of Wg and the same 64 rows of Wu, so one tile
// holds both projections of its outputs and the MMAs run as for one matrix; g
// and u then meet in shared memory, where the activation and the product are
// taken before anything is stored.
//
// Backward: dx = [dg du] [Wg; Wu], a product over the weights' rows.  A tile's
// 128 rows are half a block of columns (k), a stage is 64 weight rows.  A thread
// decodes a weight row as above (one table serves 16 codes) and stores it as
// stored, k running, which is the MMA's A operand "MN-major" in shared memory:
// the transposition costs nothing.  (Transposing the codes first, so that a lane
// could write its own column to tensor memory, took 2200 warp instructions a
// stage against 900, and 198 us instead of 110 for 512 tokens x 14336 x 4096.)
//
// With few tiles, K is split over a cluster of CTAs whose sums meet through
// distributed shared memory in a fixed order.
//
// What bounds it: at 256 tokens a tile the MMAs (512 clocks per 64 K) and the
// decode (about as long) run side by side; below, the decode alone.
//
// Every wait is bounded (about a second); on time-out the kernel records a bit
// in the device error word, drains its MMAs, frees TMEM and returns.
#include <algorithm>
#include <cstring>
#include <mutex>

#include "q2k_ffn.cuh"
#include "q2k_internal.h"
#include "q2k_tc.cuh"

namespace q2k {

__device__ unsigned int g_ffn_error;

namespace tc {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, []() {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

bool make_weight_map(CUtensorMap* map, const uint8_t* w, int N, int K, int rows) {
    const uint64_t row_bytes = static_cast<uint64_t>(K / kQK) * kBlockBytes;
    if (row_bytes % 16 != 0 || (reinterpret_cast<uintptr_t>(w) & 15) != 0) return false;
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    const cuuint64_t dims[2] = {row_bytes, static_cast<cuuint64_t>(N)};
    const cuuint64_t strides[1] = {row_bytes};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kBoxBytes), static_cast<cuuint32_t>(rows)};
    const cuuint32_t elem[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(w), dims, strides, box,
                  elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc

namespace {

using namespace tc;

constexpr int kDecWarps = 16;  // two groups of 8, one per half of a block
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kMmaWarp = kDecWarps, kWaitWarp = kDecWarps + 1, kWWarp = kDecWarps + 2,
              kXWarp0 = kDecWarps + 3;
constexpr int kThreads = 32 * (kDecWarps + 5);
constexpr int kMaxParts = 8;
constexpr int kPlanSms = 152;  // K parts are planned for the whole GPU, whatever the device
constexpr int kTileStages = 20;  // a tile's set-up and epilogue, in stages of its K loop

constexpr int kABytes = kStageK * kRows * 2;  // a decoded stage in shared memory
// Sums of a tile in shared memory: token c, row r at word 132 c + r (132: lanes
// that read two tokens apart fall on different banks).
constexpr int kSumPitch = kRows + 4;

enum class Tc { kGated, kLora, kBackward };

// Tiles of kX tokens.
// 256: two CTAs of a cluster (neighbouring row tiles) form one MMA of 256 rows
// x 256 tokens, issued by one thread of the first (cta_group::2).  Each holds
// half of the tokens' stage, so a stage is half as large and crosses from L2
// once per pair, and its ring is twice as deep in time.
// 128 and fewer: narrow MMAs issue at half the rate the tensor core takes them,
// so two threads issue, each into its own accumulator; the token ring and the A
// ring are equally deep then, and one release serves two stages of both.
template <int kX, bool kTma, Tc kMode>
struct Cfg {
    static constexpr bool kBack = kMode == Tc::kBackward;
    static constexpr bool kDuo = kX == 256;
    static constexpr int kIssuers = kDuo ? 1 : 2;
    static constexpr int kHand = kDuo || kBack ? 2 : 4;  // stages handed over at a time
    static constexpr bool kPairs = kIssuers == 2;        // stages released two at a time
    static constexpr int kHold = kDuo ? kX / 2 : kX;     // tokens of a stage in this CTA
    static constexpr int kXStage = kHold * kStageK * 2;
    static constexpr int kXStages = kDuo ? (kBack ? 8 : 12) : kBack && kX == 128 ? 6 : 8;
    static constexpr int kAStages = kBack ? (kDuo ? 4 : kXStages) : 8;
    // decoders: groups of warps on stages (backward) or block halves in turn
    static constexpr int kGroupWarps = kBack ? 4 : 8;
    static constexpr uint32_t kColA = kX * kIssuers;
    static constexpr uint32_t kTmemCols = 512;
    // raw slots: a block column of 128 weight rows, or (backward) of 64 for a
    // stage, without TMA only the 11 words of the half block that it needs
    static constexpr int kRawRows = kBack ? kStageK : kRows;
    static constexpr int kRawPitch = kTma ? kBoxBytes : kBack ? 44 : kBlockBytes;
    static constexpr int kRawBytes = kRawRows * kRawPitch;
    static constexpr int kRaw = kBack ? (kTma ? 4 : 8) : (kTma ? 2 : 3);
    // backward: decoded stages in shared memory, 64 weight rows x 128 columns
    static constexpr int kOffA = kXStages * kXStage;
    static constexpr int kOffRaw = kOffA + (kBack ? kAStages * kABytes : 0);
    // bars: x_full, x_empty [kXStages], a_full, a_empty, peer_full [kAStages],
    //       raw_full, raw_empty [kRaw], accum, drain
    static constexpr int kNumBars = 2 * kXStages + 3 * kAStages + 2 * kRaw + 2;
    static constexpr int kOffBar = (kOffRaw + kRaw * kRawBytes + 7) & ~7;
    static constexpr int kOffMisc = kOffBar + 8 * kNumBars;
    static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory");
    // the epilogue's sums, and with adapters 64 t and an id a token, reuse the rings
    static_assert(kOffBar >= (kSumPitch + (kMode == Tc::kLora ? 65 : 0)) * kX * 4, "epilogue");
    static_assert(kColA + (kBack ? 0 : 32 * kAStages) <= kTmemCols, "tensor memory");
    static_assert(kOffA % 1024 == 0 && kOffRaw % 1024 == 0, "swizzle and TMA alignment");
};

struct TcArgs {
    const uint8_t* xa;   // bf16 image of the tokens, or null: they come by the token maps
    const uint8_t* w0;   // Wg, or W
    const uint8_t* w1;   // Wu
    int M, N, K;         // N, K: the weight matrices' rows and columns
    int stages;          // 64-K stages of the whole product
    int half_stages;     // backward: those of Wg
    bool const_weights;  // the grid before does not write the weights
    bool tokens_ready;   // nor the tokens
    // gated
    void* h;
    void* gate;
    void* up;
    int act;
    // adapters
    const __nv_bfloat16* b;
    const float* t;
    const int* ids;
    void* y;             // adapters: y; backward: dx
    int R, n_adapters;
};

struct TcMaps {
    CUtensorMap w0, w1;  // weights, 112-byte boxes of 64 or 128 rows
    CUtensorMap x0, x1;  // tokens, boxes of kX rows x 64 (backward: dg and du)
};

// Stage Cp (0, 1) of one half of a block for one thread: the two K-steps of
// quant segment `seg` at shifts J = 2 Cp + {0, 1}.  qh: the thread's four quant
// words, sh: the half's two scale words shifted right by 8 seg.
template <int Cp>
__device__ __forceinline__ void decode_half_stage(const uint32_t* qh, const uint32_t* sh, float d,
                                                  float dmin, uint32_t (&o0)[8], uint32_t (&o1)[8]) {
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
        constexpr int kJ0 = 2 * Cp;
        const int j = kJ0 + jj;
        uint32_t lo, hi;
        weight_table((sh[j >> 1] >> (16 * (j & 1))) & 0xFFu, d, dmin, lo, hi);
        uint32_t* o = jj == 0 ? o0 : o1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t sel = jj == 0 ? code_selectors<kJ0>(qh[e]) : code_selectors<kJ0 + 1>(qh[e]);
            o[2 * e] = __byte_perm(lo, hi, sel);
            o[2 * e + 1] = __byte_perm(lo, hi, __umulhi(sel, 0x10000u));  // sel >> 16
        }
    }
}

// Block b of the tile's 128 rows (row r < split0 from w0, the others from w1)
// into a raw slab; rows past N are zero-filled (they decode to 0).
__device__ __forceinline__ void issue_raw(const uint8_t* w0, const uint8_t* w1, int split0,
                                          uint32_t dst, int n0, int N, size_t row_bytes, int b,
                                          int td) {
#pragma unroll 3
    for (int f = td; f < kRows * kWordsPerBlock; f += kDecThreads) {
        const int r = f / kWordsPerBlock;
        const int wd = f - r * kWordsPerBlock;
        const int n = n0 + (r < split0 ? r : r - split0);
        const bool ok = n < N;
        const uint8_t* src = (r < split0 ? w0 : w1) +
                             (ok ? static_cast<size_t>(n) * row_bytes +
                                       static_cast<size_t>(b) * kBlockBytes + 4 * wd
                                 : 0);
        cp_async_4(dst + r * kBlockBytes + 4 * wd, src, ok ? 4u : 0u);
    }
    cp_async_commit();
}

__device__ __forceinline__ void dec_barrier() {
    asm volatile("bar.sync 2, %0;" ::"n"(kDecThreads) : "memory");
}

// Adds s_a B_a t of each token's adapter to the sums: per 16 rows and eight
// tokens, one product (m16n8k16) for each adapter that occurs among them, B_a as
// stored and t split into two bf16 (16 bits); a token's sum takes only its own
// adapter's product.  Tokens [first, end), first a multiple of 8.
// t comes through shared memory 64 values a token at a time, already split: the
// two bf16 of value pair j (hi, lo) of token c at words 64 c + (2 j ^ 8 (c % 4)),
// so that the eight tokens a warp reads together fall on different banks.  B_a's
// fragments stay in registers from one token group to the next with the same
// adapter.  (Reading t and B per group from L2 took 40 us of an 85 us call: 512
// tokens, 7168 x 7168, rank 64; splitting t per group of rows 14 us; this 5 us.)
__device__ __forceinline__ void add_adapters(float* sums, uint32_t* tbuf, int* id_buf,
                                             const TcArgs& p, int n0, int m0, int first, int end) {
    const int td = threadIdx.x, warp = td >> 5, lane = td & 31;
    const int g = lane >> 2, t = lane & 3;
    const int row = 16 * (warp & 7) + g;  // this lane's rows: row, row + 8
    const bool ok0 = n0 + row < p.N, ok1 = n0 + row + 8 < p.N;
    // ids: -1 none, -2 out of range (a zero row)
    for (int c = first + td; c < end; c += kDecThreads) {
        const int id = p.ids[m0 + c];
        id_buf[c] = id < -1 || id >= p.n_adapters ? -2 : id;
    }
    for (int r0 = 0; r0 < p.R; r0 += 64) {
        const int width = min(64, p.R - r0);  // a multiple of 8
        for (int base = 16 * first + td; base < 16 * end; base += 4 * kDecThreads) {
            float4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = base + u * kDecThreads, r = 4 * (i & 15);
                v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < 16 * end && r < width)
                    v[u] = *reinterpret_cast<const float4*>(
                        p.t + static_cast<size_t>(m0 + (i >> 4)) * p.R + r0 + r);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = base + u * kDecThreads, c = i >> 4, r = 4 * (i & 15);
                if (i >= 16 * end) break;
                uint4 w;
                w.x = pack_bf16(v[u].x, v[u].y);
                w.z = pack_bf16(v[u].z, v[u].w);
                w.y = pack_bf16(v[u].x - __uint_as_float(w.x << 16),
                                v[u].y - __uint_as_float(w.x & 0xFFFF0000u));
                w.w = pack_bf16(v[u].z - __uint_as_float(w.z << 16),
                                v[u].w - __uint_as_float(w.z & 0xFFFF0000u));
                *reinterpret_cast<uint4*>(tbuf + 64 * c + (r ^ (8 * (c & 3)))) = w;
            }
        }
        dec_barrier();
        int cur = -1;
        uint32_t a[4][4];
        for (int c0 = first + 8 * (warp >> 3); c0 < end; c0 += 16) {
            const int id = c0 + g < end ? id_buf[c0 + g] : -1;
            // the ids of the columns 2 t, 2 t + 1 whose sums this lane holds
            const int id0 = __shfl_sync(0xFFFFFFFFu, id, 8 * t);
            const int id1 = __shfl_sync(0xFFFFFFFFu, id, 8 * t + 4);
            float* s0 = sums + (c0 + 2 * t) * kSumPitch + row;
            float* s1 = s0 + kSumPitch;
            if (id0 == -2) s0[0] = s0[8] = 0.f;
            if (id1 == -2) s1[0] = s1[8] = 0.f;
            unsigned todo = __ballot_sync(0xFFFFFFFFu, id >= 0);
            while (todo != 0) {
                const int ad = __shfl_sync(0xFFFFFFFFu, id, __ffs(todo) - 1);
                todo &= ~__ballot_sync(0xFFFFFFFFu, id == ad);
                if (ad != cur) {
                    cur = ad;
                    const __nv_bfloat16* b0 =
                        p.b + (static_cast<size_t>(ad) * p.N + n0 + row) * p.R + r0;
                    const __nv_bfloat16* b1 = b0 + static_cast<size_t>(8) * p.R;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        a[q][0] = a[q][1] = a[q][2] = a[q][3] = 0u;
                        const bool in0 = 16 * q < width, in1 = 16 * q + 8 < width;
                        if (ok0 && in0) a[q][0] = __ldg(reinterpret_cast<const uint32_t*>(b0 + 16 * q) + t);
                        if (ok1 && in0) a[q][1] = __ldg(reinterpret_cast<const uint32_t*>(b1 + 16 * q) + t);
                        if (ok0 && in1) a[q][2] = __ldg(reinterpret_cast<const uint32_t*>(b0 + 16 * q + 8) + t);
                        if (ok1 && in1) a[q][3] = __ldg(reinterpret_cast<const uint32_t*>(b1 + 16 * q + 8) + t);
                    }
                }
                // (four chains of two products, added at the end: a product
                // takes as long as dozens of other instructions to return)
                float e[4][4] = {};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint2 u = make_uint2(0u, 0u), v = u;
                    if (id == ad && 16 * q < width) {
                        const uint32_t* tr = tbuf + 64 * (c0 + g);
                        const int x = 8 * ((c0 + g) & 3);
                        u = *reinterpret_cast<const uint2*>(tr + ((16 * q + 2 * t) ^ x));
                        v = *reinterpret_cast<const uint2*>(tr + ((16 * q + 8 + 2 * t) ^ x));
                    }
                    if (16 * q < width) {
                        mma_bf16_16816(e[q], a[q][0], a[q][1], a[q][2], a[q][3], u.x, v.x);
                        mma_bf16_16816(e[q], a[q][0], a[q][1], a[q][2], a[q][3], u.y, v.y);
                    }
                }
                float d[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) d[c] = (e[0][c] + e[1][c]) + (e[2][c] + e[3][c]);
                if (id0 == ad) {
                    s0[0] += d[0];
                    s0[8] += d[2];
                }
                if (id1 == ad) {
                    s1[0] += d[1];
                    s1[8] += d[3];
                }
            }
        }
        dec_barrier();
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

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
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
__device__ __forceinline__ void issue_raw_rows(const TcArgs& p, uint32_t dst, int stage, int block,
                                               int half, int tg) {
    const bool up = stage >= p.half_stages;
    const int n0 = kStageK * (up ? stage - p.half_stages : stage);
    const uint8_t* w = up ? p.w1 : p.w0;
    const size_t row_bytes = static_cast<size_t>(p.K / kQK) * kBlockBytes;
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

// The weights of segment `seg` of a half block of one row at shift J: words 0..3
// of `q` -> 16 bf16 (k running).
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

template <int kX, bool kTma, Tc kMode, typename T>
__global__ void __launch_bounds__(kThreads, 1)
ffn_tc_kernel(TcArgs p, const __grid_constant__ TcMaps maps) {
    using C = Cfg<kX, kTma, kMode>;
    constexpr bool kBack = kMode == Tc::kBackward;
    constexpr bool kDuo = C::kDuo;
    constexpr int kSplit0 = kMode == Tc::kGated ? kRows / 2 : kRows;  // tile rows of w0
    extern __shared__ uint8_t smem_dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = blockIdx.x * kSplit0;  // first row of the product (backward: column k)
    const int rows = kBack ? p.K : p.N;   // rows of the product
    const int m0 = blockIdx.y * kX;
    const int tokens = min(kX, p.M - m0);
    const int nx = kDuo ? (tokens + 31) & ~31 : (tokens + 15) & ~15;  // MMA N
    // two CTAs: this one holds tokens [peer nx / 2, peer nx / 2 + nx / 2)
    const int peer = kDuo ? static_cast<int>(blockIdx.x & 1) : 0;
    const int held = kDuo ? nx / 2 : nx;
    const int m_held = m0 + peer * held;
    // K parts in whole blocks (backward: four stages, 256 weight rows)
    const int parts = gridDim.z, quads = p.stages / 4;
    const int q0 = static_cast<int>(static_cast<long>(blockIdx.z) * quads / parts);
    const int n_quads = static_cast<int>(static_cast<long>(blockIdx.z + 1) * quads / parts) - q0;
    const int n_iters = 4 * n_quads;

    const uint32_t bar_xfull = sbase + C::kOffBar;
    const uint32_t bar_xempty = bar_xfull + 8 * C::kXStages;
    const uint32_t bar_afull = bar_xempty + 8 * C::kXStages;
    const uint32_t bar_aempty = bar_afull + 8 * C::kAStages;
    const uint32_t bar_peer = bar_aempty + 8 * C::kAStages;  // (of the first CTA)
    const uint32_t bar_raw = bar_peer + 8 * C::kAStages;
    const uint32_t bar_rawempty = bar_raw + 8 * C::kRaw;
    const uint32_t bar_accum = bar_rawempty + 8 * C::kRaw;
    const uint32_t bar_drain = bar_accum + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    unsigned int* err = &g_ffn_error;

    if (warp == 0) {
        for (int s = lane; s < C::kXStages; s += 32) {
            mbar_init(bar_xfull + 8 * s, 1);   // the producer's expect-tx arrival
            mbar_init(bar_xempty + 8 * s, 1);  // MMA commit
        }
        for (int s = lane; s < C::kAStages; s += 32) {
            mbar_init(bar_afull + 8 * s, C::kGroupWarps);  // the warps of its group
            mbar_init(bar_aempty + 8 * s, C::kPairs ? C::kIssuers : 1);
            mbar_init(bar_peer + 8 * s, 1);  // the second CTA's waiter
        }
        for (int r = lane; r < C::kRaw; r += 32) {
            mbar_init(bar_raw + 8 * r, kTma ? 1 : kDecWarps);
            mbar_init(bar_rawempty + 8 * r, kBack ? C::kGroupWarps : kDecWarps);
        }
        if (lane == 0) {
            mbar_init(bar_accum, C::kIssuers);
            mbar_init(bar_drain, C::kIssuers);
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
    float* sums = reinterpret_cast<float*>(smem);

    if (warp < kDecWarps) {
        // ---------------- weight decoders ----------------
        const int td = threadIdx.x;
        const int quarter = warp & 3, sub = (warp >> 2) & 1, group = warp >> 3;
        const int row = 32 * quarter + lane;
        const uint32_t raw0 = sbase + C::kOffRaw;
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
        if (!kTma && !p.const_weights) pdl_wait_prerequisites();
        // Publish a stage decoded into two runs of eight columns of tensor memory.
        [[maybe_unused]] auto publish = [&](int i, uint32_t col0, const uint32_t (&o0)[8], uint32_t col1,
                           const uint32_t (&o1)[8]) -> bool {
            const int s = i % C::kAStages;
            const int rel = (C::kPairs ? (i | 1) : i) % C::kAStages;
            if (i >= C::kAStages &&
                !__all_sync(0xFFFFFFFFu,
                            mbar_wait_bounded(bar_aempty + 8 * rel, ((i / C::kAStages) - 1) & 1,
                                              abort_flag, err, kErrTimeoutEmpty)))
                return false;
            fence_after();  // the MMAs that read this stage are done
            tmem_store8(t_lane + C::kColA + 32u * s + col0, o0);
            tmem_store8(t_lane + C::kColA + 32u * s + col1, o1);
            tmem_store_wait();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_afull + 8 * s);
            return true;
        };
        if constexpr (kBack) {
            // group (four warps) takes every fourth stage: warp = 32 weight rows
            // and a segment, lane = the row, all four shifts
            const int own = warp >> 2, tg = td & 127;
            const int seg = warp & 1, n = 32 * ((warp >> 1) & 1) + lane;
            const int block = n0 / kQK, half = (n0 / kRows) & 1;
            if constexpr (!kTma) {
                if (own < n_iters)
                    issue_raw_rows(p, raw0 + own * C::kRawBytes, 4 * q0 + own, block, half, tg);
                else
                    cp_async_commit();
            }
            bool ok = true;  // a warp that gave up still passes the group's barriers
            for (int i = own; i < n_iters; i += 4) {
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
                    if (i + 4 < n_iters) {
                        asm volatile("bar.sync %0, 128;" ::"r"(3 + own) : "memory");
                        issue_raw_rows(p, raw0 + ((i + 4) % C::kRaw) * C::kRawBytes, 4 * q0 + i + 4,
                                       block, half, tg);
                        cp_async_wait<1>();
                    } else {
                        cp_async_wait<0>();
                    }
                    asm volatile("bar.sync %0, 128;" ::"r"(3 + own) : "memory");
                }
                if (!ok) continue;
                uint32_t q[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) q[e] = ld_shared_u32(at_q + 16 * seg + 4 * e);
                const uint32_t sc0 = ld_shared_u32(at_sc) >> (8 * seg);
                const uint32_t sc1 = ld_shared_u32(at_sc + 4) >> (8 * seg);
                const uint32_t dd = ld_shared_u32(at_d);
                if constexpr (kTma) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_rawempty + 8 * slot);
                }
                const float d = f16_bits_to_float(dd), dmin = f16_bits_to_float(dd >> 16);
                uint32_t o[4][8];
                decode_segment<0>(q, sc0 & 0xFFu, d, dmin, o[0]);
                decode_segment<1>(q, (sc0 >> 16) & 0xFFu, d, dmin, o[1]);
                decode_segment<2>(q, sc1 & 0xFFu, d, dmin, o[2]);
                decode_segment<3>(q, (sc1 >> 16) & 0xFFu, d, dmin, o[3]);
                const int s = i % C::kAStages;
                const int rel = (C::kPairs ? (i | 1) : i) % C::kAStages;
                if (i >= C::kAStages)
                    ok = __all_sync(0xFFFFFFFFu,
                                    mbar_wait_bounded(bar_aempty + 8 * rel, ((i / C::kAStages) - 1) & 1,
                                                      abort_flag, err, kErrTimeoutEmpty));
                if (!ok) continue;
                // row n of the tile: 128 bytes of columns 64 c .. at 8192 c +
                // 128 n, its 16-byte chunks swizzled by n % 8
                const uint32_t dst = sbase + C::kOffA + s * kABytes + 128 * n;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        st_shared_v4(dst + 8192 * (j >> 1) +
                                         (((4 * (j & 1) + 2 * seg + c) ^ (n & 7)) << 4),
                                     o[j][4 * c], o[j][4 * c + 1], o[j][4 * c + 2], o[j][4 * c + 3]);
                fence_async_smem();  // this thread's stores -> visible to the MMA
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_afull + 8 * s);
            }
        } else {
            const size_t row_bytes = static_cast<size_t>(p.K / kQK) * kBlockBytes;
            if constexpr (!kTma) {
                for (int b = 0; b < C::kRaw - 1; ++b) {
                    if (b < n_quads)
                        issue_raw(p.w0, p.w1, kSplit0, raw0 + b * C::kRawBytes, n0, p.N, row_bytes,
                                  q0 + b, td);
                    else
                        cp_async_commit();
                }
            }
            bool ok = true;
            for (int b = 0; b < n_quads && ok; ++b) {
                const int buf = b % C::kRaw;
                uint32_t mine = raw0 + buf * C::kRawBytes + row * C::kRawPitch;
                if constexpr (!kTma) {
                    cp_async_wait<C::kRaw - 2>();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_raw + 8 * buf);
                }
                if (!__all_sync(0xFFFFFFFFu,
                                mbar_wait_bounded(bar_raw + 8 * buf, (b / C::kRaw) & 1, abort_flag,
                                                  err, kErrTimeoutEmpty)))
                    break;
                if constexpr (kTma) {
                    mine += 4 * ((q0 + b) & 3);  // the box starts at a 16-byte boundary
                } else {
                    // every decoder has read block b - 1: its slot takes block b + kRaw - 1
                    const int nb = b + C::kRaw - 1;
                    if (nb < n_quads)
                        issue_raw(p.w0, p.w1, kSplit0, raw0 + (nb % C::kRaw) * C::kRawBytes, n0, p.N,
                                  row_bytes, q0 + nb, td);
                    else
                        cp_async_commit();
                }
                uint32_t sh[2], qh[4];
#pragma unroll
                for (int q = 0; q < 2; ++q) sh[q] = ld_shared_u32(mine + 8 * group + 4 * q) >> (8 * sub);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    qh[e] = ld_shared_u32(mine + 16 + 32 * group + 16 * sub + 4 * e);
                const uint32_t dd = ld_shared_u32(mine + 80);
                if constexpr (kTma) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_rawempty + 8 * buf);
                }
                const float d = f16_bits_to_float(dd), dmin = f16_bits_to_float(dd >> 16);
#pragma unroll
                for (int cp = 0; cp < 2; ++cp) {
                    uint32_t o0[8], o1[8];
                    if (cp == 0) decode_half_stage<0>(qh, sh, d, dmin, o0, o1);
                    else decode_half_stage<1>(qh, sh, d, dmin, o0, o1);
                    if (!publish(4 * b + 2 * group + cp, 8u * sub, o0, 8u * sub + 16u, o1)) {
                        ok = false;
                        break;
                    }
                }
            }
        }
        if constexpr (!kTma) asm volatile("cp.async.wait_all;" ::: "memory");

        // ---------------- the tile's sums to shared memory ----------------
        if (__all_sync(0xFFFFFFFFu, mbar_wait_backoff(bar_accum, 0, abort_flag, err,
                                                      kErrTimeoutAccum, 512))) {
            fence_after();
#pragma unroll 1
            for (int c0 = 16 * (warp >> 2); c0 < nx; c0 += 64) {
                float v[16];
                tmem_load16(t_lane + c0, v);
                if (C::kIssuers == 2) {
                    float u[16];
                    tmem_load16(t_lane + kX + c0, u);
#pragma unroll
                    for (int q = 0; q < 16; ++q) v[q] += u[q];
                }
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    if (c0 + q < tokens) sums[(c0 + q) * kSumPitch + row] = v[q];
            }
        }
    } else if ((warp == kMmaWarp && peer == 0) || (C::kIssuers == 2 && warp == kWaitWarp)) {
        // ---------------- MMA issuers ----------------
        // The waiter waits for the next kHand stages and meets the MMA warp at
        // named barrier 1; both pass it n_iters / kHand times whatever happens.
        // With two issuers the MMA warp takes the even stages into accumulator
        // 0, the waiter the odd ones into accumulator 1.
        const int me = warp == kMmaWarp ? 0 : 1;
        const uint32_t idesc = bf16_idesc(kDuo ? 2 * kRows : kRows, nx) | (kBack ? kIdescAMnMajor : 0u);
        const uint64_t xdesc0 = sw128_desc(sbase);
        const uint64_t adesc0 = sw128_mn_desc(sbase + C::kOffA, 8192);
        const uint32_t acc = tmem + static_cast<uint32_t>(me * kX);
        for (int i0 = 0; i0 < n_iters; i0 += C::kHand) {
            if (C::kIssuers == 2 && me == 1 && lane == 0 && !*abort_flag) {
#pragma unroll
                for (int u = 0; u < C::kHand; ++u) {
                    const int i = i0 + u;
                    if (!mbar_wait_bounded(bar_xfull + 8 * (i % C::kXStages), (i / C::kXStages) & 1,
                                           abort_flag, err, kErrTimeoutFull) ||
                        !mbar_wait_bounded(bar_afull + 8 * (i % C::kAStages), (i / C::kAStages) & 1,
                                           abort_flag, err, kErrTimeoutFull))
                        break;
                }
            }
            __syncwarp();
            asm volatile("bar.sync 1, 64;" ::: "memory");
            if (lane == 0 && !*abort_flag) {
                fence_after();
#pragma unroll
                for (int u = 0; u < C::kHand; ++u) {
                    if (C::kIssuers == 2 && (u & 1) != me) continue;
                    const int i = i0 + u;
                    const int sx = i % C::kXStages, sa = i % C::kAStages;
                    const uint64_t xdesc = xdesc0 + static_cast<uint64_t>(sx * (C::kXStage >> 4));
                    const uint32_t a_s = tmem + C::kColA + 32u * sa;
                    const uint64_t adesc = adesc0 + static_cast<uint64_t>(sa * (kABytes >> 4));
#pragma unroll
                    for (int kk = 0; kk < kStageK / 16; ++kk) {
                        const uint32_t add = i >= C::kIssuers || kk > 0;
                        if (kBack)  // (a K-step is 16 rows of 128 bytes)
                            mma_smem<kDuo>(acc, adesc + 128u * kk, xdesc + 2u * kk, idesc, add);
                        else
                            mma<kDuo>(acc, a_s + 8u * kk, xdesc + 2u * kk, idesc, add);
                    }
                    // a stage is released when a later one takes its place
                    if (C::kPairs) {
                        if ((i & ~1) + C::kAStages < n_iters)
                            commit<kDuo>(bar_aempty + 8 * ((i | 1) % C::kAStages));
                    } else {
                        if (i + C::kAStages < n_iters) commit<kDuo>(bar_aempty + 8 * sa);
                        if (i + C::kXStages < n_iters) commit<kDuo>(bar_xempty + 8 * sx);
                    }
                }
            }
            __syncwarp();
        }
        if (lane == 0) {
            if (!*abort_flag) {
                commit<kDuo>(bar_accum);
            } else {
                // no MMA may still write TMEM when it is freed
                commit<kDuo>(bar_drain);
                volatile int no_abort = 0;
                mbar_wait_bounded(bar_drain, 0, &no_abort, err, kErrTimeoutDrain);
            }
        }
        __syncwarp();
    } else if (kDuo && warp == kWaitWarp) {
        // ---------------- stage waiters of a pair of CTAs ----------------
        // The second CTA's waiter reports each of its stages to the first's,
        // which waits for both CTAs' and hands them to the MMA warp.
        for (int i0 = 0; i0 < n_iters; i0 += C::kHand) {
            if (lane == 0 && !*abort_flag) {
#pragma unroll
                for (int u = 0; u < C::kHand; ++u) {
                    const int i = i0 + u, sa = i % C::kAStages;
                    const uint32_t phase = (i / C::kAStages) & 1;
                    if (!mbar_wait_bounded(bar_xfull + 8 * (i % C::kXStages), (i / C::kXStages) & 1,
                                           abort_flag, err, kErrTimeoutFull) ||
                        !mbar_wait_bounded(bar_afull + 8 * sa, phase, abort_flag, err, kErrTimeoutFull))
                        break;
                    if (peer == 1) {
                        fence_after();
                        fence_before();
                        arrive_first_of_pair(bar_peer + 8 * sa);
                    } else if (!wait_peer_bounded(bar_peer + 8 * sa, phase, abort_flag, err,
                                                  kErrTimeoutFull)) {
                        break;
                    }
                }
            }
            __syncwarp();
            if (peer == 0) asm volatile("bar.sync 1, 64;" ::: "memory");
        }
    } else if (warp == kWWarp) {
        // ---------------- raw weight blocks ----------------
        if (kTma && lane == 0) {
            tma_prefetch_map(&maps.w0);
            if (kMode != Tc::kLora) tma_prefetch_map(&maps.w1);
            if (!p.const_weights) pdl_wait_prerequisites();
            const int n_raw = kBack ? n_iters : n_quads;
            for (int b = 0; b < n_raw; ++b) {
                const int buf = b % C::kRaw;
                if (b >= C::kRaw &&
                    !mbar_wait_bounded(bar_rawempty + 8 * buf, ((b / C::kRaw) - 1) & 1, abort_flag,
                                       err, kErrTimeoutEmpty))
                    break;
                const uint32_t dst = sbase + C::kOffRaw + buf * C::kRawBytes;
                const uint32_t bar = bar_raw + 8 * buf;
                mbar_arrive_expect_tx(bar, C::kRawBytes);
                if constexpr (kBack) {
                    const int stage = 4 * q0 + b;
                    const bool up = stage >= p.half_stages;
                    tma_load_2d(dst, up ? &maps.w1 : &maps.w0, (kBlockBytes * (n0 / kQK)) & ~15,
                                kStageK * (up ? stage - p.half_stages : stage), bar);
                } else {
                    const int x = (kBlockBytes * (q0 + b)) & ~15;
                    tma_load_2d(dst, &maps.w0, x, n0, bar);
                    if (kMode == Tc::kGated)
                        tma_load_2d(dst + kSplit0 * kBoxBytes, &maps.w1, x, n0, bar);
                }
            }
            if (*abort_flag) linger();
        }
        __syncwarp();
    } else if (warp >= kXWarp0) {
        // ---------------- token stages, even and odd ----------------
        if (lane == 0) {
            const uint8_t* src = p.xa +
                                 (static_cast<size_t>(m0 / kSuperRows) * p.stages + 4 * q0) *
                                     kSuperBytes +
                                 static_cast<size_t>(m_held % kSuperRows) * (kStageK * 2);
            const uint32_t bytes = p.xa != nullptr ? held * (kStageK * 2) : C::kXStage;
            if (p.xa == nullptr) {
                tma_prefetch_map(&maps.x0);
                if (kBack) tma_prefetch_map(&maps.x1);
            }
            if (!p.tokens_ready) {
                pdl_wait_prerequisites();  // the tokens
                pdl_allow_dependents();
            }
            for (int i = warp - kXWarp0; i < n_iters; i += 2) {
                const int s = i % C::kXStages;
                if (i >= C::kXStages &&
                    !mbar_wait_bounded(C::kPairs ? bar_aempty + 8 * ((i | 1) % C::kAStages)
                                                 : bar_xempty + 8 * s,
                                       ((i / C::kXStages) - 1) & 1, abort_flag, err, kErrTimeoutEmpty))
                    break;
                const uint32_t dst = sbase + s * C::kXStage, bar = bar_xfull + 8 * s;
                mbar_arrive_expect_tx(bar, bytes);
                if (p.xa != nullptr) {
                    bulk_copy_g2s(dst, src + static_cast<size_t>(i) * kSuperBytes, bytes, bar);
                } else {
                    // (tokens past M and, backward, weight rows past N read as zeros)
                    const int stage = 4 * q0 + i;
                    const bool up = kBack && stage >= p.half_stages;
                    tma_load_2d(dst, up ? &maps.x1 : &maps.x0,
                                kStageK * (up ? stage - p.half_stages : stage), m_held, bar);
                }
            }
            if (*abort_flag) linger();
        }
        __syncwarp();
    }

    // ---------------- epilogue ----------------
    // Every thread of every CTA of a cluster passes its barriers, whatever
    // happened before.  Part r takes its share of the tile's tokens (whole
    // groups of eight) and adds them over the parts in order; the second
    // cluster barrier keeps every part's sums alive until all are read.
    int first = 0, end = tokens;
    if (parts > 1) {  // (cluster rank: row tile of the pair + 2 part, or the part)
        const int groups = (tokens + 7) / 8, z = blockIdx.z;
        first = 8 * (z * groups / parts);
        end = min(tokens, 8 * ((z + 1) * groups / parts));
        __syncwarp();
        cluster_sync();
    } else if (warp < kDecWarps) {
        dec_barrier();
    }
    // past these barriers no wait is left that could raise the flag
    const bool done = *abort_flag == 0;
    if (warp < kDecWarps && parts > 1) {
        for (int j = first * (kRows / 4) + threadIdx.x; j < end * (kRows / 4); j += kDecThreads) {
            const int i = j / (kRows / 4) * (kSumPitch / 4) + j % (kRows / 4);
            float4 v[kMaxParts];
#pragma unroll
            for (int z = 0; z < kMaxParts; ++z)
                if (z < parts) v[z] = load_cluster4(sbase + 16 * i, kDuo ? 2 * z + peer : z);
            float4 a = v[0];
#pragma unroll
            for (int z = 1; z < kMaxParts; ++z)
                if (z < parts) {
                    a.x += v[z].x;
                    a.y += v[z].y;
                    a.z += v[z].z;
                    a.w += v[z].w;
                }
            reinterpret_cast<float4*>(sums)[i] = a;
        }
        dec_barrier();
    }
    if (warp < kDecWarps && done) {
        const bool vec = (rows & 1) == 0;  // (n0 is even: pairs are aligned)
        if constexpr (kMode == Tc::kGated) {
            // a warp takes a token at a time, a lane the rows 2 lane, 2 lane + 1
            for (int c = first + warp; c < end; c += kDecWarps) {
                const float2 g = *reinterpret_cast<const float2*>(sums + c * kSumPitch + 2 * lane);
                const float2 u =
                    *reinterpret_cast<const float2*>(sums + c * kSumPitch + kSplit0 + 2 * lane);
                const int n = n0 + 2 * lane;
                const int valid = rows - n;
                if (valid <= 0) continue;
                const size_t at = static_cast<size_t>(m0 + c) * rows + n;
                store_pair(static_cast<T*>(p.h) + at, act_value<sizeof(T) == 2>(g.x, p.act) * u.x,
                           act_value<sizeof(T) == 2>(g.y, p.act) * u.y, valid, vec);
                if (p.gate != nullptr) {
                    store_pair(static_cast<T*>(p.gate) + at, g.x, g.y, valid, vec);
                    store_pair(static_cast<T*>(p.up) + at, u.x, u.y, valid, vec);
                }
            }
        } else {
            if constexpr (kMode == Tc::kLora) {
                pdl_wait_prerequisites();  // t (written by this grid or one before)
                uint32_t* tbuf = reinterpret_cast<uint32_t*>(sums + kX * kSumPitch);
                add_adapters(sums, tbuf, reinterpret_cast<int*>(tbuf + kX * 64), p, n0, m0, first, end);
            }
            for (int c = first + warp; c < end; c += kDecWarps)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int r = 64 * q + 2 * lane;
                    const float2 v = *reinterpret_cast<const float2*>(sums + c * kSumPitch + r);
                    const int valid = rows - (n0 + r);
                    if (valid > 0)
                        store_pair(static_cast<T*>(p.y) + static_cast<size_t>(m0 + c) * rows + n0 + r,
                                   v.x, v.y, valid, vec);
                }
        }
    }
    fence_before();
    __syncwarp();
    if (kDuo || parts > 1) cluster_sync();
    else __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        tmem_free<kDuo>(tmem, C::kTmemCols);
    }
}

// x (f32 [M, K]) -> the bf16 tile image; rows past M up to a multiple of 16 are
// zeros (their sums are dropped, but the MMA reads them).  One thread writes
// 16-byte chunks, four per pass with their loads issued together.
__global__ void __launch_bounds__(256)
x_image_kernel(const float* __restrict__ x, uint8_t* __restrict__ xa, int M, int K, size_t chunks) {
    pdl_allow_dependents();
    const int per_row = K / 8, stages = K / kStageK;
    const size_t stride = static_cast<size_t>(gridDim.x) * blockDim.x;
    constexpr int kPer = 4;
    for (size_t base = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x; base < chunks;
         base += kPer * stride) {
        uint4 v[kPer];
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const size_t id = base + u * stride;
            v[u] = make_uint4(0u, 0u, 0u, 0u);
            if (id < static_cast<size_t>(M) * per_row) {
                const float4 a = __ldg(reinterpret_cast<const float4*>(x) + 2 * id);
                const float4 b = __ldg(reinterpret_cast<const float4*>(x) + 2 * id + 1);
                v[u] = make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y),
                                  pack_bf16(b.z, b.w));
            }
        }
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const size_t id = base + u * stride;
            if (id < chunks) {
                const int m = static_cast<int>(id / per_row);
                const int c = static_cast<int>(id - static_cast<size_t>(m) * per_row);
                *reinterpret_cast<uint4*>(xa + image_offset(m, c, stages)) = v[u];
            }
        }
    }
    // later grids find whatever ran before this one complete
    pdl_wait_prerequisites();
}

// dg = dh u act'(g) and du = dh act(g), rounded to bf16 as the MMA's operands:
// rows of `pitch` (the products' token matrices) and, where the caller's own
// rows are not those, of N.  A thread takes eight consecutive n of a row.
__global__ void __launch_bounds__(256)
grad_kernel(const __nv_bfloat16* __restrict__ dh, const __nv_bfloat16* __restrict__ gate,
            const __nv_bfloat16* __restrict__ up, __nv_bfloat16* __restrict__ dg,
            __nv_bfloat16* __restrict__ du, int pitch, __nv_bfloat16* __restrict__ dgate,
            __nv_bfloat16* __restrict__ dup, int M, int N, int act) {
    pdl_allow_dependents();
    const int per_row = pitch / 8;
    const bool vec = (N & 7) == 0;
    const size_t chunks = static_cast<size_t>(M) * per_row;
    for (size_t id = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x; id < chunks;
         id += static_cast<size_t>(gridDim.x) * blockDim.x) {
        const int m = static_cast<int>(id / per_row);
        const int n = 8 * static_cast<int>(id - static_cast<size_t>(m) * per_row);
        const size_t at = static_cast<size_t>(m) * N + n;
        __nv_bfloat16 h[8], g[8], u[8], a[8], b[8];
        if (vec) {
            *reinterpret_cast<uint4*>(h) = __ldg(reinterpret_cast<const uint4*>(dh + at));
            *reinterpret_cast<uint4*>(g) = __ldg(reinterpret_cast<const uint4*>(gate + at));
            *reinterpret_cast<uint4*>(u) = __ldg(reinterpret_cast<const uint4*>(up + at));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool ok = n + e < N;
                h[e] = ok ? dh[at + e] : __float2bfloat16_rn(0.f);
                g[e] = ok ? gate[at + e] : __float2bfloat16_rn(0.f);
                u[e] = ok ? up[at + e] : __float2bfloat16_rn(0.f);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float value, slope;
            act_value_slope<true>(to_float(g[e]), act, value, slope);
            a[e] = __float2bfloat16_rn(to_float(h[e]) * to_float(u[e]) * slope);
            b[e] = __float2bfloat16_rn(to_float(h[e]) * value);
        }
        const size_t to = static_cast<size_t>(m) * pitch + n;
        *reinterpret_cast<uint4*>(dg + to) = *reinterpret_cast<const uint4*>(a);
        *reinterpret_cast<uint4*>(du + to) = *reinterpret_cast<const uint4*>(b);
        if (dgate != nullptr) {
            for (int e = 0; e < 8 && n + e < N; ++e) {
                dgate[at + e] = a[e];
                dup[at + e] = b[e];
            }
        }
    }
}

// ---- plan ----------------------------------------------------------------------

struct Plan {
    int x_rows, row_tiles, token_tiles, parts;
};

// rows: those of the product's row tiles; quads: its K in parts of four stages.
// Tokens per tile: as few as hold them all up to 64.  Above, 128 or 256,
// whichever is expected to end first: waves of CTAs times stages of a K part
// times the time of a stage, about 1 : 0.7 for 256 and 128 tokens (512 tokens x
// 14336 x 4096 backwards: 110 us in tiles of 256 and two K parts, 150 us in
// tiles of 128).  K parts while the tiles leave half of the GPU or more idle.
Plan make_plan(int M, int rows, int tile_rows, int quads) {
    Plan best = {};
    double best_cost = 0;
    for (int x_rows : {32, 64, 128, 256}) {
        if (x_rows < 128 && x_rows < M) continue;
        Plan p;
        p.x_rows = x_rows;
        p.row_tiles = (rows + tile_rows - 1) / tile_rows;
        if (x_rows == 256) p.row_tiles += p.row_tiles & 1;  // pairs
        p.token_tiles = (M + x_rows - 1) / x_rows;
        const long tiles = static_cast<long>(p.row_tiles) * p.token_tiles;
        p.parts = static_cast<int>(
            std::max(1L, std::min<long>(std::min(x_rows == 256 ? kMaxParts / 2 : kMaxParts, quads),
                                        kPlanSms / tiles)));
        const long waves = (tiles * p.parts + kPlanSms - 1) / kPlanSms;
        const double stages = 4.0 * quads / p.parts;
        const double cost = waves * (stages + kTileStages) * (x_rows == 256 ? 1.0 : 0.7);
        if (best_cost == 0 || cost < best_cost) {
            best = p;
            best_cost = cost;
        }
        if (x_rows >= M) break;  // a wider tile would be empty columns
    }
    return best;
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

template <int kX, bool kTma, Tc kMode, typename T>
cudaError_t launch_tc_as(const TcArgs& a, const Plan& plan, const TcMaps& maps, int device,
                         cudaStream_t stream) {
    using C = Cfg<kX, kTma, kMode>;
    static bool attr_done[64] = {};
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[device]) {
        const cudaError_t e = cudaFuncSetAttribute(ffn_tc_kernel<kX, kTma, kMode, T>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   C::kSmemBytes);
        if (e != cudaSuccess) return e;
        attr_done[device] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(plan.row_tiles, plan.token_tiles, plan.parts);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (C::kDuo || plan.parts > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = C::kDuo ? 2 : 1;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = static_cast<unsigned>(plan.parts);
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, ffn_tc_kernel<kX, kTma, kMode, T>, a, maps);
}

// T: the type of the results.  x0, x1: bf16 token matrices [M, x_cols] with rows
// `x_pitch` apart (x1: backward, du), or null with a.xa an image.
template <Tc kMode, typename T>
cudaError_t launch_tc(const TcArgs& a, const Plan& plan, const void* x0, const void* x1, int x_cols,
                      int x_pitch, int device, cudaStream_t stream) {
    alignas(64) TcMaps maps;
    memset(&maps, 0, sizeof maps);
    const int rows = kMode == Tc::kLora ? kRows : 64;
    const bool tma = make_weight_map(&maps.w0, a.w0, a.N, a.K, rows) &&
                     (kMode == Tc::kLora || make_weight_map(&maps.w1, a.w1, a.N, a.K, rows));
    const int held = std::min(plan.x_rows, 128);  // tokens of a stage in one CTA
    if (a.xa == nullptr &&
        (!make_token_map(&maps.x0, x0, a.M, x_cols, x_pitch, held) ||
         (kMode == Tc::kBackward && !make_token_map(&maps.x1, x1, a.M, x_cols, x_pitch, held))))
        return cudaErrorNotSupported;
#define Q2K_TC_CASE(X)                                                              \
    case X:                                                                         \
        return tma ? launch_tc_as<X, true, kMode, T>(a, plan, maps, device, stream) \
                   : launch_tc_as<X, false, kMode, T>(a, plan, maps, device, stream);
    switch (plan.x_rows) {
        Q2K_TC_CASE(32)
        Q2K_TC_CASE(64)
        Q2K_TC_CASE(128)
        Q2K_TC_CASE(256)
    }
#undef Q2K_TC_CASE
    return cudaErrorInvalidValue;
}

size_t image_bytes(int M, int K) {
    return static_cast<size_t>((M + kSuperRows - 1) / kSuperRows) * kSuperRows * K * 2;
}

// x W^T: bf16 tokens go to the kernel by their own tensor map, f32 tokens by an
// image.  behind_grid: one of this call's own grids (which does not write x) is
// before, and lets its dependents start only when x is complete.
template <Tc kMode>
cudaError_t launch_forward(TcArgs a, bool bf16, const void* x, void* workspace, int device,
                           int sm_count, bool behind_grid, cudaStream_t stream) {
    const Plan plan = make_plan(a.M, a.N, kMode == Tc::kGated ? 64 : kRows, a.K / kQK);
    a.stages = a.K / kStageK;
    a.tokens_ready = bf16 && behind_grid;
    if (bf16)
        return launch_tc<kMode, __nv_bfloat16>(a, plan, x, nullptr, a.K, a.K, device, stream);
    a.xa = static_cast<const uint8_t*>(workspace);
    // the image's grid started when all before it was complete: the weights are
    a.const_weights = true;
    const size_t chunks = static_cast<size_t>((a.M + 15) & ~15) * (a.K / 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<size_t>((chunks + 255) / 256, sm_count * 4)));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = behind_grid ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, x_image_kernel, static_cast<const float*>(x),
                                             static_cast<uint8_t*>(workspace), a.M, a.K, chunks);
    if (e != cudaSuccess) return e;
    return launch_tc<kMode, float>(a, plan, nullptr, nullptr, 0, 0, device, stream);
}

// Columns of dg and du as the product's K: whole parts of two stages each.
int backward_cols(int N) { return (N + 2 * kStageK - 1) / (2 * kStageK) * (2 * kStageK); }
// Their rows' pitch: the caller's own when those are whole 16 bytes.
int backward_pitch(int N) { return (N + 7) & ~7; }

}  // namespace

size_t gated_tc_workspace_bytes(const GatedArgs& a) { return a.bf16 ? 0 : image_bytes(a.M, a.K); }

cudaError_t launch_gated_tc(const GatedArgs& a, void* workspace, cudaStream_t stream) {
    TcArgs t = {};
    t.w0 = a.wg;
    t.w1 = a.wu;
    t.M = a.M;
    t.N = a.N;
    t.K = a.K;
    t.const_weights = a.const_weights;
    t.h = a.h;
    t.gate = a.gate;
    t.up = a.up;
    t.act = a.act;
    return launch_forward<Tc::kGated>(t, a.bf16, a.x, workspace, a.device, a.sm_count, false, stream);
}

size_t lora_tc_workspace_bytes(const LoraArgs& a) { return a.bf16 ? 0 : image_bytes(a.M, a.K); }

cudaError_t launch_lora_tc(const LoraArgs& a, const float* t, void* workspace, cudaStream_t stream) {
    TcArgs c = {};
    c.w0 = c.w1 = a.w;
    c.M = a.M;
    c.N = a.N;
    c.K = a.K;
    c.const_weights = true;  // the grid before started when all before it was complete
    c.b = a.b;
    c.t = t;
    c.ids = a.ids;
    c.y = a.y;
    c.R = a.R;
    c.n_adapters = a.n_adapters;
    return launch_forward<Tc::kLora>(c, a.bf16, a.x, workspace, a.device, a.sm_count, true, stream);
}

// Workspace: dg and du, unless the caller takes them in rows of whole 16 bytes.
static bool backward_in_place(const GatedBackwardArgs& a) {
    return a.dgate != nullptr && backward_pitch(a.N) == a.N;
}
static size_t backward_matrix_bytes(const GatedBackwardArgs& a) {
    return (static_cast<size_t>(a.M) * backward_pitch(a.N) * 2 + 255) & ~size_t(255);
}
size_t gated_backward_workspace_bytes(const GatedBackwardArgs& a) {
    return backward_in_place(a) ? 0 : 2 * backward_matrix_bytes(a);
}

cudaError_t launch_gated_backward(const GatedBackwardArgs& a, void* workspace, cudaStream_t stream) {
    const int pitch = backward_pitch(a.N), cols = backward_cols(a.N);
    const bool own = backward_in_place(a);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    __nv_bfloat16* dg = own ? a.dgate : reinterpret_cast<__nv_bfloat16*>(ws);
    __nv_bfloat16* du = own ? a.dup
                            : reinterpret_cast<__nv_bfloat16*>(ws + backward_matrix_bytes(a));
    const size_t chunks = static_cast<size_t>(a.M) * (pitch / 8);
    const unsigned blocks =
        static_cast<unsigned>(std::min<size_t>((chunks + 255) / 256, static_cast<size_t>(a.sm_count) * 8));
    grad_kernel<<<blocks, 256, 0, stream>>>(a.dh, a.gate, a.up, dg, du, pitch,
                                            own ? nullptr : a.dgate, own ? nullptr : a.dup, a.M, a.N,
                                            a.act);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    TcArgs t = {};
    t.w0 = a.wg;
    t.w1 = a.wu;
    t.M = a.M;
    t.N = a.N;
    t.K = a.K;
    t.const_weights = true;  // the grid before started when all before it was complete
    t.half_stages = cols / kStageK;
    t.stages = 2 * t.half_stages;
    t.y = a.dx;
    const Plan plan = make_plan(a.M, a.K, kRows, t.stages / 4);
    return launch_tc<Tc::kBackward, __nv_bfloat16>(t, plan, dg, du, a.N, pitch, a.device, stream);
}

cudaError_t read_and_clear_ffn_error(uint32_t* out, cudaStream_t stream) {
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_ffn_error, sizeof(unsigned int), 0,
                                              cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbolAsync(g_ffn_error, &zero, sizeof(unsigned int), 0,
                                    cudaMemcpyHostToDevice, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    return e;
}

}  // namespace q2k
