// Many tokens times Q2_K weights on the tensor cores (tcgen05): the gated
// feed-forward block, and a projection with low-rank adapters.
//
// A prepass writes x as bf16 in the swizzled tile image that the MMA reads.  A
// CTA then computes 128 weight rows x up to 256 tokens over K: 16 warps decode
// Q2_K blocks into tensor memory (the MMA's A operand: one weight row per
// lane), x stages arrive by bulk copies (the B operand), and f32 sums build up
// in tensor memory.  For the gated block the 128 rows are 64 rows of Wg and the
// same 64 rows of Wu, so one tile holds both projections of its outputs and the
// MMAs run as for a single matrix; g and u then meet in shared memory, where
// the activation and the product are taken before anything is stored.
// With few tiles, K is split over CTAs whose sums the last one to finish adds
// in a fixed order.
//
// What bounds it: at 256 tokens a tile the MMAs (512 clocks per 64 weights of
// K) and the decode (about as long) run side by side; below, the decode alone,
// whatever the tokens.
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

// Tiles of kX tokens.  256: one accumulator, one thread issues the MMAs.  128
// and fewer: narrow MMAs issue at half the rate the tensor core takes them, so
// two threads issue, each into its own accumulator; x and A rings are equally
// deep, and one release serves a pair of stages of both.
template <int kX, bool kTma>
struct Cfg {
    static constexpr int kIssuers = kX == 256 ? 1 : 2;
    static constexpr int kHand = kX == 256 ? 2 : 4;  // stages handed to the issuers at a time
    static constexpr bool kPairs = kIssuers == 2;    // stages released in pairs
    static constexpr int kXStage = kX * kStageK * 2;
    static constexpr int kXStages = kX == 256 ? 6 : 8;
    static constexpr int kAStages = 8;
    static constexpr uint32_t kColA = kX * kIssuers;
    static constexpr uint32_t kTmemCols = 512;
    static constexpr int kRawBytes = kRows * (kTma ? kBoxBytes : kBlockBytes);
    static constexpr int kRaw = kTma ? 2 : 3;        // raw blocks in flight
    static constexpr int kOffRaw = kXStages * kXStage;
    // bars: x_full, x_empty [kXStages], a_full, a_empty [kAStages], raw_full,
    //       raw_empty [kRaw], accum, drain
    static constexpr int kNumBars = 2 * kXStages + 2 * kAStages + 2 * kRaw + 2;
    static constexpr int kOffBar = (kOffRaw + kRaw * kRawBytes + 7) & ~7;
    static constexpr int kOffMisc = kOffBar + 8 * kNumBars;
    static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
    static_assert(kOffRaw >= kRows * kX * 4, "the sums of a tile reuse the x ring");
    static_assert(kColA + 32 * kAStages <= kTmemCols, "tensor memory");
    static_assert(kOffRaw % 1024 == 0, "TMA destination alignment");
};

struct TcArgs {
    const uint8_t* xa;  // x image
    const uint8_t* w0;  // gated: Wg; else W
    const uint8_t* w1;  // gated: Wu
    int M, N, K;
    float* partial;     // [tile][part][token][128], with more than one part
    unsigned int* tile_count;
    // gated
    void* h;
    void* gate;
    void* up;
    int act;
    // adapters
    const __nv_bfloat16* b;
    const float* t;
    const int* ids;
    void* y;
    int R, n_adapters;
};

enum class Tc { kGated, kLora };

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

// Sums of a tile in shared memory: token c, row r at word 128 c + r.  Adds
// s_a B_a t of each token's adapter: per 16 rows and eight tokens, one product
// (m16n8k16) for each adapter that occurs among them, B_a as stored and t split
// into two bf16 (16 bits); a token's sum takes only its own adapter's product.
__device__ __forceinline__ void add_adapters(float* sums, const TcArgs& p, int n0, int m0,
                                             int tokens, int warp, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int row = 16 * (warp & 7) + g;  // this lane's rows: row, row + 8
    const bool ok0 = n0 + row < p.N, ok1 = n0 + row + 8 < p.N;
    for (int c0 = 8 * (warp >> 3); c0 < tokens; c0 += 16) {
        const int m = m0 + c0 + g;  // column g of the product
        int id = c0 + g < tokens ? p.ids[m] : -1;
        const bool bad = id < -1 || id >= p.n_adapters;
        if (bad) id = -1;
        // the ids of the columns 2 t, 2 t + 1 whose sums this lane holds
        const int id0 = __shfl_sync(0xFFFFFFFFu, id, 8 * t);
        const int id1 = __shfl_sync(0xFFFFFFFFu, id, 8 * t + 4);
        const int bad0 = __shfl_sync(0xFFFFFFFFu, int(bad), 8 * t);
        const int bad1 = __shfl_sync(0xFFFFFFFFu, int(bad), 8 * t + 4);
        float* s0 = sums + (c0 + 2 * t) * kRows + row;
        float* s1 = s0 + kRows;
        if (bad0) s0[0] = s0[8] = 0.f;  // an id out of range: a zero row
        if (bad1) s1[0] = s1[8] = 0.f;
        unsigned todo = __ballot_sync(0xFFFFFFFFu, id >= 0);
        while (todo != 0) {
            const int a = __shfl_sync(0xFFFFFFFFu, id, __ffs(todo) - 1);
            todo &= ~__ballot_sync(0xFFFFFFFFu, id == a);
            const __nv_bfloat16* b0 = p.b + (static_cast<size_t>(a) * p.N + n0 + row) * p.R;
            const __nv_bfloat16* b1 = b0 + static_cast<size_t>(8) * p.R;
            const float* tr = p.t + static_cast<size_t>(m) * p.R;
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            for (int r = 0; r < p.R; r += 16) {
                // K slots 2 t, 2 t + 1 and 2 t + 8, 2 t + 9 of the step
                uint32_t a0 = 0, a1 = 0, a2 = 0, a3 = 0, h0 = 0, h1 = 0, l0 = 0, l1 = 0;
                const bool wide = r + 8 < p.R;  // (the rank is a multiple of 8)
                if (ok0) {
                    a0 = __ldg(reinterpret_cast<const uint32_t*>(b0 + r) + t);
                    if (wide) a2 = __ldg(reinterpret_cast<const uint32_t*>(b0 + r + 8) + t);
                }
                if (ok1) {
                    a1 = __ldg(reinterpret_cast<const uint32_t*>(b1 + r) + t);
                    if (wide) a3 = __ldg(reinterpret_cast<const uint32_t*>(b1 + r + 8) + t);
                }
                if (id == a) {
                    const float2 u = reinterpret_cast<const float2*>(tr + r)[t];
                    h0 = pack_bf16(u.x, u.y);
                    l0 = pack_bf16(u.x - __uint_as_float(h0 << 16),
                                   u.y - __uint_as_float(h0 & 0xFFFF0000u));
                    if (wide) {
                        const float2 v = reinterpret_cast<const float2*>(tr + r + 8)[t];
                        h1 = pack_bf16(v.x, v.y);
                        l1 = pack_bf16(v.x - __uint_as_float(h1 << 16),
                                       v.y - __uint_as_float(h1 & 0xFFFF0000u));
                    }
                }
                mma_bf16_16816(d, a0, a1, a2, a3, h0, h1);
                mma_bf16_16816(d, a0, a1, a2, a3, l0, l1);
            }
            if (id0 == a) {
                s0[0] += d[0];
                s0[8] += d[2];
            }
            if (id1 == a) {
                s1[0] += d[1];
                s1[8] += d[3];
            }
        }
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

template <int kX, bool kTma, Tc kMode, typename T>
__global__ void __launch_bounds__(kThreads, 1)
ffn_tc_kernel(TcArgs p, const __grid_constant__ CUtensorMap map0,
              const __grid_constant__ CUtensorMap map1) {
    using C = Cfg<kX, kTma>;
    constexpr int kSplit0 = kMode == Tc::kGated ? kRows / 2 : kRows;  // tile rows of w0
    constexpr int kRawDepth = C::kRaw, kRawBytes = C::kRawBytes;
    extern __shared__ uint8_t smem_dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = blockIdx.x * kSplit0;
    const int m0 = blockIdx.y * kX;
    const int tokens = min(kX, p.M - m0);
    const int nx = (tokens + 15) & ~15;  // MMA N
    const int blocks = p.K / kQK;
    const size_t row_bytes = static_cast<size_t>(blocks) * kBlockBytes;
    const int parts = gridDim.z;
    const int kb0 = static_cast<int>(static_cast<long>(blockIdx.z) * blocks / parts);
    const int n_blocks = static_cast<int>(static_cast<long>(blockIdx.z + 1) * blocks / parts) - kb0;
    const int n_iters = 4 * n_blocks;

    const uint32_t bar_xfull = sbase + C::kOffBar;
    const uint32_t bar_xempty = bar_xfull + 8 * C::kXStages;
    const uint32_t bar_afull = bar_xempty + 8 * C::kXStages;
    const uint32_t bar_aempty = bar_afull + 8 * C::kAStages;
    const uint32_t bar_raw = bar_aempty + 8 * C::kAStages;
    const uint32_t bar_rawempty = bar_raw + 8 * C::kRaw;
    const uint32_t bar_accum = bar_rawempty + 8 * C::kRaw;
    const uint32_t bar_drain = bar_accum + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    volatile int* last_part = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
    unsigned int* err = &g_ffn_error;

    if (warp == 0) {
        for (int s = lane; s < C::kXStages; s += 32) {
            mbar_init(bar_xfull + 8 * s, 1);   // the producer's expect-tx arrival
            mbar_init(bar_xempty + 8 * s, 1);  // MMA commit
        }
        for (int s = lane; s < C::kAStages; s += 32) {
            mbar_init(bar_afull + 8 * s, kDecWarps / 2);  // the warps of its group
            mbar_init(bar_aempty + 8 * s, C::kPairs ? C::kIssuers : 1);
        }
        for (int r = lane; r < C::kRaw; r += 32) {
            mbar_init(bar_raw + 8 * r, kTma ? 1 : kDecWarps);
            mbar_init(bar_rawempty + 8 * r, kDecWarps);
        }
        if (lane == 0) {
            mbar_init(bar_accum, C::kIssuers);
            mbar_init(bar_drain, C::kIssuers);
            *abort_flag = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);

    if (warp < kDecWarps) {
        // ---------------- weight decoders ----------------
        const int td = threadIdx.x;
        const int quarter = warp & 3, seg = (warp >> 2) & 1, half = warp >> 3;
        const int row = 32 * quarter + lane;
        const uint32_t raw0 = sbase + C::kOffRaw;
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
        const uint32_t a_col0 = t_lane + C::kColA + 8u * seg;
        if constexpr (!kTma) {
            for (int b = 0; b < kRawDepth - 1; ++b) {
                if (b < n_blocks)
                    issue_raw(p.w0, p.w1, kSplit0, raw0 + b * kRawBytes, n0, p.N, row_bytes, kb0 + b, td);
                else
                    cp_async_commit();
            }
        }
        bool ok = true;
        for (int b = 0; b < n_blocks && ok; ++b) {
            const int buf = b % kRawDepth;
            uint32_t mine;
            if constexpr (!kTma) {
                cp_async_wait<kRawDepth - 2>();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_raw + 8 * buf);
            }
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar_raw + 8 * buf, (b / kRawDepth) & 1,
                                                           abort_flag, err, kErrTimeoutEmpty)))
                break;
            if constexpr (kTma) {
                // the box starts at the 16-byte boundary at or below the block
                mine = raw0 + buf * kRawBytes + row * kBoxBytes + 4 * ((kb0 + b) & 3);
            } else {
                // every decoder has read block b - 1: its slab takes block b + depth - 1
                const int nb = b + kRawDepth - 1;
                if (nb < n_blocks)
                    issue_raw(p.w0, p.w1, kSplit0, raw0 + (nb % kRawDepth) * kRawBytes, n0, p.N,
                              row_bytes, kb0 + nb, td);
                else
                    cp_async_commit();
                mine = raw0 + buf * kRawBytes + row * kBlockBytes;
            }
            uint32_t sh[2], qh[4];
#pragma unroll
            for (int q = 0; q < 2; ++q) sh[q] = ld_shared_u32(mine + 8 * half + 4 * q) >> (8 * seg);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                qh[e] = ld_shared_u32(mine + 16 + 32 * half + 16 * seg + 4 * e);
            const uint32_t dd = ld_shared_u32(mine + 80);
            if constexpr (kTma) {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_rawempty + 8 * buf);
            }
            const float d = f16_bits_to_float(dd), dmin = f16_bits_to_float(dd >> 16);
#pragma unroll
            for (int cp = 0; cp < 2; ++cp) {
                const int i = 4 * b + 2 * half + cp;
                const int s = i % C::kAStages;
                uint32_t o0[8], o1[8];
                if (cp == 0) decode_half_stage<0>(qh, sh, d, dmin, o0, o1);
                else decode_half_stage<1>(qh, sh, d, dmin, o0, o1);
                const int rel = (C::kPairs ? (i | 1) : i) % C::kAStages;
                if (i >= C::kAStages &&
                    !__all_sync(0xFFFFFFFFu,
                                mbar_wait_bounded(bar_aempty + 8 * rel, ((i / C::kAStages) - 1) & 1,
                                                  abort_flag, err, kErrTimeoutEmpty))) {
                    ok = false;
                    break;
                }
                fence_after();  // the MMAs that read this stage are done
                tmem_store8(a_col0 + 32u * s, o0);
                tmem_store8(a_col0 + 32u * s + 16u, o1);
                tmem_store_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_afull + 8 * s);
            }
        }
        if constexpr (!kTma) asm volatile("cp.async.wait_all;" ::: "memory");

        // ---------------- epilogue ----------------
        const bool done = __all_sync(
            0xFFFFFFFFu, mbar_wait_backoff(bar_accum, 0, abort_flag, err, kErrTimeoutAccum, 512));
        float* sums = reinterpret_cast<float*>(smem);  // token c, row r at word 128 c + r
        const size_t tile = static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x;
        float* part0 = p.partial + tile * parts * (kX * kRows);
        if (done) {
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
                float* dst = parts == 1 ? sums : part0 + blockIdx.z * (kX * kRows);
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    if (c0 + q < tokens) dst[(c0 + q) * kRows + row] = v[q];
            }
        }
        // (a CTA that timed out still takes part in every barrier and count;
        // past this barrier no wait is left that could raise the flag)
        dec_barrier();
        bool mine_to_store = *abort_flag == 0;
        if (parts > 1) {
            // The part that counts last adds the parts in order.  The barrier
            // and the fence order every thread's stores before the count; the
            // second fence orders the count before the loads.
            if (td == 0) {
                __threadfence();
                pdl_wait_prerequisites();  // the prepass zeroed the counts
                const unsigned prev = atomicAdd(&p.tile_count[tile], 1u);
                __threadfence();
                *last_part = prev == static_cast<unsigned>(parts) - 1u;
            }
            dec_barrier();
            mine_to_store = *last_part != 0;
            if (mine_to_store) {
                const int quads = tokens * (kRows / 4);
                for (int i = td; i < quads; i += kDecThreads) {
                    float4 v[kMaxParts];
#pragma unroll
                    for (int z = 0; z < kMaxParts; ++z)
                        if (z < parts)
                            v[z] = __ldcg(reinterpret_cast<const float4*>(part0 + z * (kX * kRows)) + i);
                    float4 s = v[0];
#pragma unroll
                    for (int z = 1; z < kMaxParts; ++z)
                        if (z < parts) {
                            s.x += v[z].x;
                            s.y += v[z].y;
                            s.z += v[z].z;
                            s.w += v[z].w;
                        }
                    reinterpret_cast<float4*>(sums)[i] = s;
                }
            }
            dec_barrier();
        }
        if (mine_to_store) {
            const bool vec = (p.N & 1) == 0;  // (n0 is even: pairs are aligned)
            if constexpr (kMode == Tc::kGated) {
                // a warp takes a token at a time, a lane the rows 2 lane, 2 lane + 1
                for (int c = warp; c < tokens; c += kDecWarps) {
                    const float2 g = *reinterpret_cast<const float2*>(sums + c * kRows + 2 * lane);
                    const float2 u =
                        *reinterpret_cast<const float2*>(sums + c * kRows + kSplit0 + 2 * lane);
                    const int n = n0 + 2 * lane;
                    const int valid = p.N - n;
                    if (valid <= 0) continue;
                    const size_t at = static_cast<size_t>(m0 + c) * p.N + n;
                    store_pair(static_cast<T*>(p.h) + at, act_value(g.x, p.act) * u.x,
                               act_value(g.y, p.act) * u.y, valid, vec);
                    if (p.gate != nullptr) {
                        store_pair(static_cast<T*>(p.gate) + at, g.x, g.y, valid, vec);
                        store_pair(static_cast<T*>(p.up) + at, u.x, u.y, valid, vec);
                    }
                }
            } else {
                // (t is written before the image, whose grid waited for it)
                pdl_wait_prerequisites();
                add_adapters(sums, p, n0, m0, tokens, warp, lane);
                dec_barrier();
                for (int c = warp; c < tokens; c += kDecWarps)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int r = 64 * q + 2 * lane;
                        const float2 v = *reinterpret_cast<const float2*>(sums + c * kRows + r);
                        const int valid = p.N - (n0 + r);
                        if (valid > 0)
                            store_pair(static_cast<T*>(p.y) + static_cast<size_t>(m0 + c) * p.N + n0 + r,
                                       v.x, v.y, valid, vec);
                    }
            }
        }
    } else if (warp == kMmaWarp || (C::kIssuers == 2 && warp == kWaitWarp)) {
        // ---------------- MMA issuers ----------------
        // The waiter waits for the next kHand stages and meets the MMA warp at
        // named barrier 1; both pass it n_iters / kHand times whatever happens.
        // With two issuers the MMA warp takes the even stages into accumulator
        // 0, the waiter the odd ones into accumulator 1.
        const int me = warp == kMmaWarp ? 0 : 1;
        const uint32_t idesc = bf16_idesc(nx);
        const uint64_t xdesc0 = sw128_desc(sbase);
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
#pragma unroll
                    for (int kk = 0; kk < kStageK / 16; ++kk)
                        mma(acc, a_s + 8u * kk, xdesc + 2u * kk, idesc, i >= C::kIssuers || kk > 0);
                    // a stage is released when a later one takes its place
                    if (C::kPairs) {
                        if ((i & ~1) + C::kAStages < n_iters)
                            commit(bar_aempty + 8 * ((i | 1) % C::kAStages));
                    } else {
                        if (i + C::kAStages < n_iters) commit(bar_aempty + 8 * sa);
                        commit(bar_xempty + 8 * sx);
                    }
                }
            }
            __syncwarp();
        }
        if (lane == 0) {
            if (!*abort_flag) {
                commit(bar_accum);
            } else {
                // no MMA may still write TMEM when it is freed
                commit(bar_drain);
                volatile int no_abort = 0;
                mbar_wait_bounded(bar_drain, 0, &no_abort, err, kErrTimeoutDrain);
            }
        }
        __syncwarp();
    } else if (warp == kWaitWarp) {
        // ---------------- stage waiter of a single issuer ----------------
        for (int i0 = 0; i0 < n_iters; i0 += C::kHand) {
            if (lane == 0 && !*abort_flag) {
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
        }
    } else if (warp == kWWarp) {
        // ---------------- raw weight blocks ----------------
        if (kTma && lane == 0) {
            tma_prefetch_map(&map0);
            if (kSplit0 < kRows) tma_prefetch_map(&map1);
            for (int b = 0; b < n_blocks; ++b) {
                const int buf = b % kRawDepth;
                if (b >= kRawDepth &&
                    !mbar_wait_bounded(bar_rawempty + 8 * buf, ((b / kRawDepth) - 1) & 1, abort_flag,
                                       err, kErrTimeoutEmpty))
                    break;
                const uint32_t dst = sbase + C::kOffRaw + buf * kRawBytes;
                const int x = (kBlockBytes * (kb0 + b)) & ~15;
                mbar_arrive_expect_tx(bar_raw + 8 * buf, kRawBytes);
                tma_load_2d(dst, &map0, x, n0, bar_raw + 8 * buf);
                if (kSplit0 < kRows)
                    tma_load_2d(dst + kSplit0 * kBoxBytes, &map1, x, n0, bar_raw + 8 * buf);
            }
            if (*abort_flag) linger();
        }
        __syncwarp();
    } else {
        // ---------------- x stages, even and odd ----------------
        if (lane == 0) {
            const uint8_t* src = p.xa +
                                 (static_cast<size_t>(m0 / kSuperRows) * (p.K / kStageK) + 4 * kb0) *
                                     kSuperBytes +
                                 static_cast<size_t>(m0 % kSuperRows) * (kStageK * 2);
            const uint32_t bytes = static_cast<uint32_t>(nx) * (kStageK * 2);
            pdl_wait_prerequisites();  // the image
            pdl_allow_dependents();
            for (int i = warp - kXWarp0; i < n_iters; i += 2) {
                const int s = i % C::kXStages;
                if (i >= C::kXStages &&
                    !mbar_wait_bounded(C::kPairs ? bar_aempty + 8 * ((i | 1) % C::kAStages)
                                                 : bar_xempty + 8 * s,
                                       ((i / C::kXStages) - 1) & 1, abort_flag, err, kErrTimeoutEmpty))
                    break;
                mbar_arrive_expect_tx(bar_xfull + 8 * s, bytes);
                bulk_copy_g2s(sbase + s * C::kXStage, src + static_cast<size_t>(i) * kSuperBytes,
                              bytes, bar_xfull + 8 * s);
            }
            if (*abort_flag) linger();
        }
        __syncwarp();
    }

    fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        tmem_free(tmem, C::kTmemCols);
    }
}

// x [M, K] -> the bf16 tile image; rows past M up to a multiple of 16 are zeros
// (they are MMA columns whose sums are dropped, but a NaN there would be read).
// One thread writes one 16-byte chunk.  Also zeroes the tile counts.
template <typename T>
__global__ void __launch_bounds__(256)
x_image_kernel(const T* __restrict__ x, uint8_t* __restrict__ xa, int M, int K, size_t chunks,
               unsigned int* __restrict__ tile_count, int tiles) {
    pdl_allow_dependents();
    const int per_row = K / 8, stages = K / kStageK;
    const size_t stride = static_cast<size_t>(gridDim.x) * blockDim.x;
    for (size_t t = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x; t < tiles; t += stride)
        tile_count[t] = 0u;
    constexpr int kPer = 4;  // chunks per pass, their loads issued together
    for (size_t base = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x; base < chunks;
         base += kPer * stride) {
        uint4 v[kPer];
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const size_t id = base + u * stride;
            v[u] = make_uint4(0u, 0u, 0u, 0u);
            if (id < static_cast<size_t>(M) * per_row) {
                if constexpr (sizeof(T) == 2) {
                    v[u] = __ldg(reinterpret_cast<const uint4*>(x) + id);
                } else {
                    const float4 a = __ldg(reinterpret_cast<const float4*>(x) + 2 * id);
                    const float4 b = __ldg(reinterpret_cast<const float4*>(x) + 2 * id + 1);
                    v[u] = make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y),
                                      pack_bf16(b.z, b.w));
                }
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

// ---- plan ----------------------------------------------------------------------

// Tokens per tile: as few as hold them all up to 128; 256 (each decoded weight
// then serves twice the MMA work) once tiles of 128 would take more than one
// wave of CTAs.
int tile_tokens(int M, int row_tiles) {
    if (M <= 32) return 32;
    if (M <= 64) return 64;
    const long ctas = static_cast<long>(row_tiles) * ((M + 127) / 128);
    return ctas > kPlanSms ? 256 : 128;
}

struct Plan {
    int x_rows, row_tiles, token_tiles, parts;
    size_t image, partial, counts;  // bytes
};

Plan make_plan(int M, int N, int K, bool gated) {
    Plan p;
    const int rows = gated ? kRows / 2 : kRows;
    p.row_tiles = (N + rows - 1) / rows;
    p.x_rows = tile_tokens(M, p.row_tiles);
    p.token_tiles = (M + p.x_rows - 1) / p.x_rows;
    const long tiles = static_cast<long>(p.row_tiles) * p.token_tiles;
    // K parts while the tiles leave half of the GPU or more idle
    p.parts = static_cast<int>(std::max(1L, std::min<long>(std::min(kMaxParts, K / kQK), kPlanSms / tiles)));
    const size_t m_pad = static_cast<size_t>((M + kSuperRows - 1) / kSuperRows) * kSuperRows;
    p.image = m_pad * K * 2;
    p.partial = p.parts > 1 ? static_cast<size_t>(tiles) * p.parts * p.x_rows * kRows * 4 : 0;
    p.counts = p.parts > 1 ? ((static_cast<size_t>(tiles) * 4 + 255) & ~size_t(255)) : 0;
    return p;
}

size_t plan_bytes(const Plan& p) { return p.image + p.partial + p.counts; }

template <int kX, bool kTma, Tc kMode, typename T>
cudaError_t launch_tc_as(const TcArgs& a, const Plan& plan, const CUtensorMap& m0,
                         const CUtensorMap& m1, int device, cudaStream_t stream) {
    using C = Cfg<kX, kTma>;
    constexpr int kSmem = C::kSmemBytes;
    static_assert(kSmem <= 232448, "shared memory");
    static bool attr_done[64] = {};
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[device]) {
        const cudaError_t e = cudaFuncSetAttribute(ffn_tc_kernel<kX, kTma, kMode, T>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        attr_done[device] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(plan.row_tiles, plan.token_tiles, plan.parts);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, ffn_tc_kernel<kX, kTma, kMode, T>, a, m0, m1);
}

template <Tc kMode, typename T>
cudaError_t launch_tc(TcArgs a, const T* x, void* workspace, int device, int sm_count,
                      bool behind_grid, cudaStream_t stream) {
    const Plan plan = make_plan(a.M, a.N, a.K, kMode == Tc::kGated);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.xa = ws;
    a.partial = reinterpret_cast<float*>(ws + plan.image);
    a.tile_count = reinterpret_cast<unsigned int*>(ws + plan.image + plan.partial);
    const size_t chunks = static_cast<size_t>((a.M + 15) & ~15) * (a.K / 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<size_t>((chunks + 255) / 256, sm_count * 4)));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    // behind one of this call's own grids (which does not write x) the prepass
    // may start early; otherwise it starts when all before it is complete
    cfg.numAttrs = behind_grid ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, x_image_kernel<T>, x, ws, a.M, a.K, chunks,
                                       a.tile_count,
                                       plan.parts > 1 ? plan.row_tiles * plan.token_tiles : 0);
    if (e != cudaSuccess) return e;
    alignas(64) CUtensorMap m0, m1;
    memset(&m0, 0, sizeof m0);
    memset(&m1, 0, sizeof m1);
    const int rows = kMode == Tc::kGated ? kRows / 2 : kRows;
    const bool tma = make_weight_map(&m0, a.w0, a.N, a.K, rows) &&
                     (kMode != Tc::kGated || make_weight_map(&m1, a.w1, a.N, a.K, rows));
#define Q2K_TC_CASE(X)                                                                          \
    case X:                                                                                     \
        return tma ? launch_tc_as<X, true, kMode, T>(a, plan, m0, m1, device, stream)           \
                   : launch_tc_as<X, false, kMode, T>(a, plan, m0, m1, device, stream);
    switch (plan.x_rows) {
        Q2K_TC_CASE(32)
        Q2K_TC_CASE(64)
        Q2K_TC_CASE(128)
        Q2K_TC_CASE(256)
    }
#undef Q2K_TC_CASE
    return cudaErrorInvalidValue;
}

}  // namespace

size_t gated_tc_workspace_bytes(const GatedArgs& a) {
    return plan_bytes(make_plan(a.M, a.N, a.K, true));
}

cudaError_t launch_gated_tc(const GatedArgs& a, void* workspace, cudaStream_t stream) {
    TcArgs t = {};
    t.w0 = a.wg;
    t.w1 = a.wu;
    t.M = a.M;
    t.N = a.N;
    t.K = a.K;
    t.h = a.h;
    t.gate = a.gate;
    t.up = a.up;
    t.act = a.act;
    if (a.bf16)
        return launch_tc<Tc::kGated>(t, static_cast<const __nv_bfloat16*>(a.x), workspace, a.device,
                                     a.sm_count, false, stream);
    return launch_tc<Tc::kGated>(t, static_cast<const float*>(a.x), workspace, a.device, a.sm_count,
                                 false, stream);
}

size_t lora_tc_workspace_bytes(const LoraArgs& a) {
    return plan_bytes(make_plan(a.M, a.N, a.K, false));
}

cudaError_t launch_lora_tc(const LoraArgs& a, const float* t, void* workspace, cudaStream_t stream) {
    TcArgs c = {};
    c.w0 = c.w1 = a.w;
    c.M = a.M;
    c.N = a.N;
    c.K = a.K;
    c.b = a.b;
    c.t = t;
    c.ids = a.ids;
    c.y = a.y;
    c.R = a.R;
    c.n_adapters = a.n_adapters;
    if (a.bf16)
        return launch_tc<Tc::kLora>(c, static_cast<const __nv_bfloat16*>(a.x), workspace, a.device,
                                    a.sm_count, true, stream);
    return launch_tc<Tc::kLora>(c, static_cast<const float*>(a.x), workspace, a.device, a.sm_count,
                                true, stream);
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
