// Few tokens times Q2_K weights with exact weights (m <= 16 bf16 or 8 f32
// tokens a pass): the gated feed-forward block and the projection with
// adapters of a decode step.
//
// A call reads each weight byte once and does little with it, so the bound is
// HBM; what can keep a kernel from it is the decode arithmetic.  A block's dot
// product is
//     sum_k w x = d * sum_g sc_g sum_l q x  -  dmin * sum_g m_g X_g,
// X_g the sum of x over group g (16 weights), sc and m 4-bit, q 2-bit.  The
// inner sums multiply small integers: q sc (at most 45) is exact in f16, and a
// 2-bit code masked in place out of a quant word already is an f16 (a
// subnormal, q 2^(2j-24) at shift 2j).  One AND and one packed multiply by sc
// thus give two exact weights, where forming dl q - ml in f32 takes three
// instructions for each; the tensor cores (m16n8k16, f16 in, f32 sums) take the
// products of 16 rows, 16 weights and 8 columns of x at once.  d and dmin enter
// once per block, in f32.
//
// x goes to f16 per (token, block), scaled by a power of two so that the
// block's largest |x| lies in [2^10, 2^11): a bf16 x is then exact down to 2^-27
// of that largest value, and an f32 x is two columns, x' = hi + lo, exact to 22
// bits.  X_g is summed in f32 and enters as hi + lo as well.
//
// Work split: a CTA's warps divide the K blocks of a row among themselves and
// keep their blocks' x in registers for every row; a unit of 32 weight rows
// (16 gate and the same 16 up rows, or 32 rows of W) streams through each warp's
// own ring of 84-byte block columns (cp.async), and the warps' sums meet in
// shared memory in a fixed order.
#include <cuda_runtime.h>

#include <algorithm>

#include "q2k_device.cuh"
#include "q2k_ffn.cuh"
#include "q2k_internal.h"

namespace q2k {

namespace {

constexpr int kWarps = 16;
constexpr int kDepth = 5;             // block columns in flight per warp
constexpr int kUnitRows = 16;         // rows of an MMA tile; a unit has two tiles
// Row r of an item starts at word 21 r + 28 (r / 4): the eight rows and four
// 16-byte slices that a warp reads together then fall on 32 different banks.
constexpr int kItemBytes = 4 * 4 * 112;
constexpr int kGroupUnits = 8;        // units whose sums are kept when K takes several passes

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    const __half2 v = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    const __half2 v = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// A thread's 64 values of one block of x as loaded (j: shift, 16 values each).
template <typename T>
struct RawX {
    uint4 v[4][sizeof(T) == 4 ? 4 : 2];
    __device__ __forceinline__ void load(const T* p, bool ok) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < (sizeof(T) == 4 ? 4 : 2); ++q)
                v[j][q] = ok ? __ldg(reinterpret_cast<const uint4*>(p + 32 * j) + q)
                             : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void get(int j, float (&f)[16]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f[4 * q] = __uint_as_float(v[j][q].x);
                f[4 * q + 1] = __uint_as_float(v[j][q].y);
                f[4 * q + 2] = __uint_as_float(v[j][q].z);
                f[4 * q + 3] = __uint_as_float(v[j][q].w);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint32_t w[4] = {v[j][q].x, v[j][q].y, v[j][q].z, v[j][q].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[8 * q + 2 * e] = __uint_as_float(w[e] << 16);
                    f[8 * q + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
                }
            }
        }
    }
};

// One block of x for eight columns (B fragments of its 16 weight steps and of
// the group sums), and the powers of two that undo its scaling for the two
// columns a thread holds of a product.  Lane (g, t): column g, the 64 weights
// 128 (t / 2) + 16 (t % 2) + 32 j + l.  Step (i, j) takes lanes l = 4 i .. 4 i + 3
// of shift j.  Columns: tokens (bf16), or token c / 2's hi and lo part (f32).
template <typename T>
struct XBlock {
    uint32_t x[32];   // step 4 i + j: {l = 4i, 4i + 2}, {4i + 1, 4i + 3}
    uint32_t s[4];    // group sums: hi {0, 2}, {1, 3}; lo (bf16 only) the same
    float undo[2];
};

template <typename T>
__device__ __forceinline__ void load_x_block(const T* x, int K, int block, int m0, int M, int lane,
                                             XBlock<T>& o) {
    constexpr bool kSplit = sizeof(T) == 4;
    const int g = lane >> 2, t = lane & 3;
    const int token = m0 + (kSplit ? g >> 1 : g);
    const T* p = x + static_cast<size_t>(token) * K + 256 * block + 128 * (t >> 1) + 16 * (t & 1);
    RawX<T> raw;
    raw.load(p, token < M);
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float v[16];
        raw.get(j, v);
#pragma unroll
        for (int l = 0; l < 16; ++l) top = fmaxf(top, fabsf(v[l]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    // 2^(10 - e), e the exponent of the block's largest |x| (at least -100, so
    // that the power is finite; smaller blocks keep their zeros and f32 range)
    const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 10 - e) << 23);
    const float down = __uint_as_float(static_cast<uint32_t>(127 - 10 + e) << 23);
    const bool lo_part = kSplit && (g & 1);
    float sum[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float v[16];
        raw.get(j, v);
        sum[j] = 0.f;
#pragma unroll
        for (int l = 0; l < 16; ++l) {
            v[l] *= up;
            sum[j] += v[l];
            if (kSplit) {
                const float hi = __half2float(__float2half_rn(v[l]));
                v[l] = lo_part ? v[l] - hi : hi;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o.x[2 * (4 * i + j)] = pack_f16x2(v[4 * i], v[4 * i + 2]);
            o.x[2 * (4 * i + j) + 1] = pack_f16x2(v[4 * i + 1], v[4 * i + 3]);
        }
    }
    float lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float hi = __half2float(__float2half_rn(sum[j]));
        lo[j] = sum[j] - hi;
        sum[j] = lo_part ? lo[j] : hi;
    }
    o.s[0] = pack_f16x2(sum[0], sum[2]);
    o.s[1] = pack_f16x2(sum[1], sum[3]);
    o.s[2] = pack_f16x2(lo[0], lo[2]);
    o.s[3] = pack_f16x2(lo[1], lo[3]);
    // a thread's product columns are 2 t and 2 t + 1: columns held by lanes
    // 4 (2 t) and 4 (2 t + 1)
    o.undo[0] = __shfl_sync(0xFFFFFFFFu, down, 8 * t);
    o.undo[1] = __shfl_sync(0xFFFFFFFFu, down, 8 * t + 4);
}

struct RowWords {
    uint32_t q[4];
    uint32_t sc;  // the slice's four scale bytes, shift 0 first
    uint32_t dd;
};

__device__ __forceinline__ RowWords read_row(uint32_t row, int t) {
    RowWords r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.q[i] = ld_shared_u32(row + 16 + 16 * t + 4 * i);
    const uint32_t s0 = ld_shared_u32(row + 8 * (t >> 1)), s1 = ld_shared_u32(row + 8 * (t >> 1) + 4);
    r.sc = __byte_perm(s0, s1, t & 1 ? 0x7531u : 0x6420u);
    r.dd = ld_shared_u32(row + 80);
    return r;
}

// The scales of a slice as packed f16 sc_j 2^(5 - 2j): the nibble under the
// exponent byte of 2^(15 - 2j), less that power.
__device__ __forceinline__ void scale_pairs(uint32_t sc, uint32_t (&s)[4]) {
    const uint32_t n = sc & 0x0F0F0F0Fu;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t sel = static_cast<uint32_t>(0x0101 * (j | ((4 + j) << 4)));
        const uint32_t base = 0x78007800u - 0x08000800u * j;
        s[j] = hsub2(__byte_perm(n, 0x60687078u, sel), base);
    }
}

// One block of 16 weight rows (rows g and g + 8 of this lane) times NT columns
// of eight: acc += d sum q sc x - dmin sum m X, scaled back.
template <typename T, int NT>
__device__ __forceinline__ void block_product(uint32_t item, int lane, const XBlock<T> (&x)[NT],
                                              float (&acc)[NT][4]) {
    const int g = lane >> 2, t = lane & 3;
    const uint32_t row = item + 84 * (g & 3) + 448 * (g >> 2);
    const RowWords a = read_row(row, t), b = read_row(row + 896, t);
    uint32_t sa[4], sb[4];
    scale_pairs(a.sc, sa);
    scale_pairs(b.sc, sb);
    float d[NT][4], e[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) d[n][c] = e[n][c] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a1 = a.q[i] >> 8, b1 = b.q[i] >> 8;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t mask = 0x00030003u << (2 * j);
            const uint32_t w0 = hmul2(a.q[i] & mask, sa[j]), w1 = hmul2(b.q[i] & mask, sb[j]);
            const uint32_t w2 = hmul2(a1 & mask, sa[j]), w3 = hmul2(b1 & mask, sb[j]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                mma_f16(d[n], w0, w1, w2, w3, x[n].x[2 * (4 * i + j)], x[n].x[2 * (4 * i + j) + 1]);
        }
    }
    // minima: nibble m at bit 4 of its byte is the f16 m 2^-20
    const uint32_t m0 = a.sc & 0x00F000F0u, m1 = b.sc & 0x00F000F0u;
    const uint32_t m2 = (a.sc >> 8) & 0x00F000F0u, m3 = (b.sc >> 8) & 0x00F000F0u;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        mma_f16(e[n], m0, m1, m2, m3, x[n].s[0], x[n].s[1]);
        if (sizeof(T) == 2) mma_f16(e[n], m0, m1, m2, m3, x[n].s[2], x[n].s[3]);
    }
    // q sc carries 2^-19, m carries 2^-20
    const float da = f16_bits_to_float(a.dd) * 0x1p19f, db = f16_bits_to_float(b.dd) * 0x1p19f;
    const float ma = f16_bits_to_float(a.dd >> 16) * -0x1p20f;
    const float mb = f16_bits_to_float(b.dd >> 16) * -0x1p20f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        acc[n][0] = fmaf(x[n].undo[0], fmaf(ma, e[n][0], da * d[n][0]), acc[n][0]);
        acc[n][1] = fmaf(x[n].undo[1], fmaf(ma, e[n][1], da * d[n][1]), acc[n][1]);
        acc[n][2] = fmaf(x[n].undo[0], fmaf(mb, e[n][2], db * d[n][2]), acc[n][2]);
        acc[n][3] = fmaf(x[n].undo[1], fmaf(mb, e[n][3], db * d[n][3]), acc[n][3]);
    }
}

struct RowsArgs {
    const uint8_t* w0;    // tiles 0 and 1 of a unit: rows from unit * unit_step on
    const uint8_t* w1;
    int unit_step;        // rows from one unit to the next
    int tile1_row;        // first row of tile 1 within the unit's rows of w1
    int M, N, K;
    int units;            // units of weight rows
    int kw;               // warps that share K
    int groups;           // row groups of kw warps in a CTA
    int passes;           // passes over K
    bool const_weights;
    bool x_ready;         // the grid before does not write x
    // gated
    void* h;
    void* gate;
    void* up;
    int act;
    // adapters
    const __nv_bfloat16* b;
    const float* t;       // [m][R], scaled
    const int* ids;
    void* y;
    int R, n_adapters;
};

enum class Rows { kGated, kLora };

__device__ __forceinline__ void cp_async_word(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}

template <typename T, int NT, int S, Rows kMode>
__global__ void __launch_bounds__(kWarps * 32, 1) rows_kernel(const T* __restrict__ x, RowsArgs p) {
    constexpr bool kSplit = sizeof(T) == 4;
    constexpr int kTokens = NT * (kSplit ? 4 : 8);  // tokens of a pass
    constexpr int kFrag = NT * (kSplit ? 2 : 4);    // a thread's sums of one tile
    constexpr int kOut = 32 * kFrag;                // sums of one tile
    extern __shared__ __align__(16) uint8_t smem[];
    // (a shuffle tells the compiler that the warp's index is uniform)
    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const int group = warp / p.kw, kw = warp - group * p.kw;
    pdl_allow_dependents();
    if (group >= p.groups) return;  // (no barrier counts these warps)
    const int m0 = blockIdx.y * kTokens;
    const int blocks = p.K / kQK;
    const size_t row_bytes = static_cast<size_t>(blocks) * kBlockBytes;
    const uint32_t ring = smem_u32(smem) + warp * kDepth * kItemBytes;
    // sums of the group's warps, two buffers; then sums kept over passes
    float* red = reinterpret_cast<float*>(smem + kWarps * kDepth * kItemBytes) +
                 static_cast<size_t>(group) * p.kw * 2 * (2 * kOut);
    float* kept = reinterpret_cast<float*>(smem + kWarps * kDepth * kItemBytes) +
                  kWarps * 2 * (2 * kOut);
    const int workers = gridDim.x * p.groups;
    const int worker = blockIdx.x * p.groups + group;
    const int my_units = worker < p.units ? (p.units - 1 - worker) / workers + 1 : 0;
    const int per_pass = (blocks + p.passes - 1) / p.passes;
    const int group_threads = 32 * p.kw;
    const int gt = kw * 32 + lane;  // thread within the group

    bool waited = false;
    for (int u0 = 0; u0 < my_units; u0 += (p.passes > 1 ? kGroupUnits : my_units)) {
        const int u1 = p.passes > 1 ? min(my_units, u0 + kGroupUnits) : my_units;
        for (int pass = 0; pass < p.passes; ++pass) {
            const int b0 = pass * per_pass;
            const int b1 = min(blocks, b0 + per_pass);
            const int first = b0 + kw * S;                      // this warp's blocks
            const int slots = max(0, min(S, b1 - first));
            const int items = (u1 - u0) * slots * 2;
            // item i: unit u0 + i / (2 slots), slot (i / 2) % slots, tile i % 2
            int iu = u0, is = 0, it = 0, issued = 0;
            auto issue = [&]() {
                if (issued < items) {
                    const int unit = worker + iu * workers;
                    const int row0 = unit * p.unit_step + (it ? p.tile1_row : 0);
                    const uint8_t* src = (it ? p.w1 : p.w0) + static_cast<size_t>(row0) * row_bytes +
                                         static_cast<size_t>(first + is) * kBlockBytes;
                    const uint32_t dst = ring + (issued % kDepth) * kItemBytes + 4 * lane;
                    const int valid = p.N - row0;
                    // one row per copy, a word per lane; rows past N read as
                    // zero bytes (d = dmin = 0)
                    if (lane < kWordsPerBlock) {
                        if (valid >= kUnitRows) {
#pragma unroll
                            for (int r = 0; r < kUnitRows; ++r)
                                cp_async_word(dst + 84 * r + 112 * (r >> 2),
                                              src + static_cast<size_t>(r) * row_bytes + 4 * lane, 4u);
                        } else {
#pragma unroll 1
                            for (int r = 0; r < kUnitRows; ++r)
                                cp_async_word(dst + 84 * r + 112 * (r >> 2),
                                              r < valid ? src + static_cast<size_t>(r) * row_bytes + 4 * lane
                                                        : p.w0,
                                              r < valid ? 4u : 0u);
                        }
                    }
                    ++issued;
                    if (++it == 2) {
                        it = 0;
                        if (++is == slots) {
                            is = 0;
                            ++iu;
                        }
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            if (!waited && !p.const_weights) {
                pdl_wait_prerequisites();
                waited = true;
            }
#pragma unroll
            for (int i = 0; i < kDepth - 1; ++i) issue();
            if (!waited && !p.x_ready) {
                pdl_wait_prerequisites();
                waited = true;
            }
            XBlock<T> xb[S][NT];
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (s < slots)
                        load_x_block(x, p.K, first + s, m0 + n * (kTokens / NT), p.M, lane, xb[s][n]);
            int item = 0;
            for (int u = u0; u < u1; ++u) {
                float acc[2][NT][4];
#pragma unroll
                for (int a = 0; a < 2; ++a)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[a][n][c] = 0.f;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    if (s >= slots) break;
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
                        // item's words are in; the item before is read by all lanes
                        __syncwarp();
                        issue();
                        block_product<T, NT>(ring + (item % kDepth) * kItemBytes, lane, xb[s], acc[a]);
                        ++item;
                    }
                }
                // this warp's sums, in fragment order
                float* mine = red + (static_cast<size_t>(u & 1) * p.kw + kw) * (2 * kOut);
#pragma unroll
                for (int a = 0; a < 2; ++a)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (kSplit) {  // hi and lo columns of a token
                            mine[a * kOut + (2 * n) * 32 + lane] = acc[a][n][0] + acc[a][n][1];
                            mine[a * kOut + (2 * n + 1) * 32 + lane] = acc[a][n][2] + acc[a][n][3];
                        } else {
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                mine[a * kOut + (4 * n + c) * 32 + lane] = acc[a][n][c];
                        }
                    }
                asm volatile("bar.sync %0, %1;" ::"r"(group), "r"(group_threads) : "memory");
                const bool last = pass == p.passes - 1;
                if (kMode == Rows::kLora && last && !waited) {
                    pdl_wait_prerequisites();  // t
                    waited = true;
                }
                const float* all = red + static_cast<size_t>(u & 1) * p.kw * (2 * kOut);
                const int unit = worker + u * workers;
                for (int o = gt; o < kOut; o += group_threads) {
                    float v[2] = {0.f, 0.f};
                    for (int w = 0; w < p.kw; ++w) {
                        v[0] += all[w * (2 * kOut) + o];
                        v[1] += all[w * (2 * kOut) + kOut + o];
                    }
                    if (p.passes > 1) {
                        float* k = kept + (u - u0) * (2 * kOut) + o;
                        if (pass > 0) {
                            v[0] += k[0];
                            v[1] += k[kOut];
                        }
                        if (!last) {
                            k[0] = v[0];
                            k[kOut] = v[1];
                            continue;
                        }
                    }
                    const int f = o >> 5, l = o & 31;
                    // fragment f of lane l: its row of the tile and its token
                    const int r = (l >> 2) + 8 * (kSplit ? f & 1 : (f >> 1) & 1);
                    const int m = m0 + (kSplit ? (f >> 1) * 4 + (l & 3)
                                               : (f >> 2) * 8 + 2 * (l & 3) + (f & 1));
                    const int n = unit * p.unit_step + r;
                    if (m >= p.M) continue;
                    if (kMode == Rows::kGated) {
                        if (n >= p.N) continue;
                        const size_t at = static_cast<size_t>(m) * p.N + n;
                        static_cast<T*>(p.h)[at] = from_float<T>(act_value<!kSplit>(v[0], p.act) * v[1]);
                        if (p.gate != nullptr) {
                            static_cast<T*>(p.gate)[at] = from_float<T>(v[0]);
                            static_cast<T*>(p.up)[at] = from_float<T>(v[1]);
                        }
                    } else {
                        const int id = p.ids[m];
                        const bool has = id >= 0 && id < p.n_adapters;
#pragma unroll
                        for (int a = 0; a < 2; ++a) {
                            const int na = n + a * p.tile1_row;
                            if (na >= p.N) continue;
                            if (has) {
                                const uint4* br = reinterpret_cast<const uint4*>(
                                    p.b + (static_cast<size_t>(id) * p.N + na) * p.R);
                                const float4* tr = reinterpret_cast<const float4*>(
                                    p.t + static_cast<size_t>(m) * p.R);
                                for (int c = 0; c < p.R / 8; ++c) {
                                    const uint4 bv = __ldg(br + c);
                                    const float4 t0 = tr[2 * c], t1 = tr[2 * c + 1];
                                    const uint32_t bw[4] = {bv.x, bv.y, bv.z, bv.w};
                                    const float tv[8] = {t0.x, t0.y, t0.z, t0.w,
                                                         t1.x, t1.y, t1.z, t1.w};
#pragma unroll
                                    for (int q = 0; q < 4; ++q) {
                                        v[a] = fmaf(__uint_as_float(bw[q] << 16), tv[2 * q], v[a]);
                                        v[a] = fmaf(__uint_as_float(bw[q] & 0xFFFF0000u),
                                                    tv[2 * q + 1], v[a]);
                                    }
                                }
                            } else if (id != -1) {
                                v[a] = 0.f;  // an id out of range: a zero row
                            }
                            static_cast<T*>(p.y)[static_cast<size_t>(m) * p.N + na] =
                                from_float<T>(v[a]);
                        }
                    }
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            // a next pass reuses both sum buffers from its first unit on
            asm volatile("bar.sync %0, %1;" ::"r"(group), "r"(group_threads) : "memory");
        }
    }
    if (!waited) pdl_wait_prerequisites();
}

template <typename T, int NT, int S, Rows kMode>
cudaError_t launch_as(const void* x, RowsArgs& p, int device, int sm_count, cudaStream_t stream) {
    constexpr int kTokens = NT * (sizeof(T) == 4 ? 4 : 8);
    constexpr int kOut = 32 * NT * (sizeof(T) == 4 ? 2 : 4);
    constexpr int kSmem = kWarps * kDepth * kItemBytes + kWarps * 2 * 2 * kOut * 4 +
                          kGroupUnits * 2 * kOut * 4;
    static_assert(kSmem <= 232448, "shared memory");
    static bool attr_done[64] = {};
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[device]) {
        const cudaError_t e = cudaFuncSetAttribute(rows_kernel<T, NT, S, kMode>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        attr_done[device] = true;
    }
    const int blocks = p.K / kQK;
    p.passes = (blocks + kWarps * S - 1) / (kWarps * S);
    const int per_pass = (blocks + p.passes - 1) / p.passes;
    p.kw = (per_pass + S - 1) / S;
    p.groups = p.passes > 1 ? 1 : kWarps / p.kw;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::min(sm_count, (p.units + p.groups - 1) / p.groups),
                       (p.M + kTokens - 1) / kTokens);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rows_kernel<T, NT, S, kMode>, static_cast<const T*>(x), p);
}

// Columns of x in registers: one tile of eight and up to two blocks a warp, or
// two tiles (more than 8 bf16 or 4 f32 tokens) and one block.
template <typename T, Rows kMode>
cudaError_t launch_rows_mode(const void* x, RowsArgs& p, int device, int sm_count,
                             cudaStream_t stream) {
    if (p.M > (sizeof(T) == 4 ? 4 : 8))
        return launch_as<T, 2, 1, kMode>(x, p, device, sm_count, stream);
    if (p.K / kQK > kWarps) return launch_as<T, 1, 2, kMode>(x, p, device, sm_count, stream);
    return launch_as<T, 1, 1, kMode>(x, p, device, sm_count, stream);
}

}  // namespace

cudaError_t launch_gated_rows(const GatedArgs& a, cudaStream_t stream) {
    RowsArgs p = {};
    p.w0 = a.wg;
    p.w1 = a.wu;
    p.unit_step = kUnitRows;
    p.tile1_row = 0;
    p.M = a.M;
    p.N = a.N;
    p.K = a.K;
    p.units = (a.N + kUnitRows - 1) / kUnitRows;
    p.const_weights = a.const_weights;
    p.h = a.h;
    p.gate = a.gate;
    p.up = a.up;
    p.act = a.act;
    return a.bf16 ? launch_rows_mode<__nv_bfloat16, Rows::kGated>(a.x, p, a.device, a.sm_count, stream)
                  : launch_rows_mode<float, Rows::kGated>(a.x, p, a.device, a.sm_count, stream);
}

cudaError_t launch_lora_rows(const LoraArgs& a, const float* t, cudaStream_t stream) {
    RowsArgs p = {};
    p.w0 = p.w1 = a.w;
    p.unit_step = 2 * kUnitRows;
    p.tile1_row = kUnitRows;
    p.M = a.M;
    p.N = a.N;
    p.K = a.K;
    p.units = (a.N + 2 * kUnitRows - 1) / (2 * kUnitRows);
    p.const_weights = a.const_weights;
    p.x_ready = true;
    p.b = a.b;
    p.t = t;
    p.ids = a.ids;
    p.y = a.y;
    p.R = a.R;
    p.n_adapters = a.n_adapters;
    return a.bf16 ? launch_rows_mode<__nv_bfloat16, Rows::kLora>(a.x, p, a.device, a.sm_count, stream)
                  : launch_rows_mode<float, Rows::kLora>(a.x, p, a.device, a.sm_count, stream);
}

}  // namespace q2k
