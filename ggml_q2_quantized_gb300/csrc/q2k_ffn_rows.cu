// Few tokens times Q2_K weights with exact weights (m <= 16 bf16 or 8 f32
// tokens a pass): the gated feed-forward block and the projection with
// adapters of a decode step.
//
// A call reads each weight byte once and does little with it, so the floor is
// HBM's; what keeps a kernel from it is the arithmetic.  A block's dot product is
//     sum_k w x = d * sum_g sc_g sum_l q x  -  dmin * sum_g m_g X_g,
// X_g the sum of x over group g (16 weights), sc and m 4-bit, q 2-bit.  The
// inner sums multiply small integers: q sc (at most 45) is exact in f16, and a
// 2-bit code masked in place out of a quant word already is an f16 (a
// subnormal, q 2^(2j-24) at shift 2j).  One AND and one packed multiply by sc
// thus give two exact weights, where forming dl q - ml in f32 takes three
// instructions for each; the tensor cores (m16n8k16, f16 in, f32 sums) take the
// products of 16 rows, 16 weights and 8 columns of x at once.  d and dmin enter
// once per block, in f32.  The two matrices of 14336 x 4096 take 21.2 us with 16 bf16
// tokens and 16.5 with up to 8 (HBM alone would take 5.7): with the products left out
// (36 a block of 16 rows with 16 tokens) 11.8 us are left, with the multiplies by sc
// left out 19.0; the tensor pipe is busy for a third of the time, issue for a half.
//
// A single token has its products in integers instead, four weights an
// instruction (dp4a): 13.6 us, 8.1 with them left out (4.6 TB/s of weights
// for longer matrices).  Its x is rounded to 22 bits beside its block's largest
// (XBytes below), coarser than the two f16 parts.
//
// x goes to f16 per (token, block), scaled by a power of two so that the
// block's largest |x| lies in [2^10, 2^11): a bf16 x is then exact down to 2^-27
// of that largest value, and an f32 x is two columns, x' = hi + lo, exact to 22
// bits.  X_g is summed in f32 and enters as hi + lo as well.
//
// Two kernels: stream_kernel (below) where a row's blocks suit its bulk copies, and
// rows_kernel for the rest: up to 8 blocks, more than 16 that are no multiple of
// four or more than 128, or weights off 16 bytes.
//
// Work split of rows_kernel: a CTA's warps divide the K blocks of a row among themselves and
// keep their blocks' x in registers for every row; a unit of 32 weight rows
// (16 gate and the same 16 up rows, or 32 rows of W) streams through each warp's
// own ring of 84-byte block columns (cp.async), and the warps' sums meet in
// shared memory in a fixed order.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "q2k_device.cuh"
#include "q2k_ffn.cuh"
#include "q2k_internal.h"
#include "q2k_tc.cuh"

namespace q2k {

namespace {

constexpr int kWarps = 16;
constexpr int kDepth = 5;             // block columns in flight per warp
constexpr int kUnitRows = 16;         // rows of an MMA tile; a unit has two tiles
// Row r of an item starts at word 21 r + 28 (r / 4): the eight rows and four
// 16-byte slices that a warp reads together then fall on 32 different banks.
constexpr int kItemBytes = 4 * 4 * 112;
constexpr int kMaxRowParts = 8;       // (the largest portable cluster)
constexpr int kMaxDepth = 8;          // units in flight of a streaming CTA
constexpr size_t kMaxSmem = 227 * 1024;
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
__device__ __forceinline__ void block_product(const RowWords& a, const RowWords& b,
                                              const XBlock<T> (&x)[NT], float (&acc)[NT][4]) {
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

// One block of one token as integers, for the slice t of each row that a lane has:
// x 2^(21 - e), e the exponent of the block's largest |x|, rounded to 22 bits and
// sign, its three digits in a word each for four weights that lie in one quant word
// at one shift; and the digits of the group sums X_g of the slice's four shifts.
// Digits are signed bytes, so that a small x has small digits and its products lose
// nothing beside a large one's.  The rounding is 2^-22 of the largest |x| (none for
// a bf16 x down to 2^-14 of it).  A block most of whose values matter little beside
// its largest would lose much of those: where more than a quarter of them are below
// 2^-9 of it, what the rounding left goes through the same products as 22 bits more
// (the block is `wide`; of 20 000 blocks of normal values none is, nor of silu(g) u
// with g and u of deviation 1 or 1.5, and one in 40 at 4).  14336 x 4096: 13.6 us
// without such blocks, 4 us more with one of the 16, 13 with all.  These products
// stand in a loop of their own: beside the ordinary ones they cost every call 1 us.
struct XBytes {
    uint32_t x[4][3][4];  // shift, digit, quant word
    uint32_t s[4];
    __device__ __forceinline__ uint4 quad(int j, int d) const {
        return make_uint4(x[j][d][0], x[j][d][1], x[j][d][2], x[j][d][3]);
    }
    __device__ __forceinline__ uint4 sums() const { return make_uint4(s[0], s[1], s[2], s[3]); }
};
constexpr int kXWords = 4 * (3 * 16 + 4);  // a block's, in shared memory
constexpr float kRest = 0x1p-22f;          // the unit of the rest's integers, in x's
// The same, left in shared memory.
struct StoredXBytes {
    const uint4* at;
    __device__ __forceinline__ uint4 quad(int j, int d) const { return at[3 * j + d]; }
    __device__ __forceinline__ uint4 sums() const { return at[12]; }
};

// Eight values times `scale` as integers w, what their rounding left in `rest`.
__device__ __forceinline__ void split_integers(const float (&v)[8], float scale, uint32_t (&w)[8],
                                               float (&rest)[8]) {
#pragma unroll
    for (int l = 0; l < 8; ++l) {
        // 1.5 2^23 + an integer of at most 2^21 or 2^22: its low bits are that
        // integer's; v times a power of two and the difference are exact
        const float u = v[l] * scale, big = u + 12582912.f;
        w[l] = __float_as_uint(big) - 0x4B400000u;
        rest[l] = u - (big - 12582912.f);
    }
}

// A lane's integers (eight weights of slice t at shift g / 2, words 2 (g % 2) ..)
// into the block's words in shared memory.
__device__ __forceinline__ void store_digits(const uint32_t (&n)[8], int lane, uint32_t* buf) {
    const int g = lane >> 2, t = lane & 3, j = g >> 1, half = g & 1;
    uint32_t w[8];
    int sum = 0;
#pragma unroll
    for (int l = 0; l < 8; ++l) {
        sum += static_cast<int>(n[l]);
        w[l] = (n[l] + 0x00808080u) ^ 0x00808080u;  // signed digits
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint32_t* a = w + 4 * q;
        const uint32_t p01 = __byte_perm(a[0], a[1], 0x5140u), p23 = __byte_perm(a[2], a[3], 0x5140u);
        const uint32_t h01 = __byte_perm(a[0], a[1], 0x0062u), h23 = __byte_perm(a[2], a[3], 0x0062u);
        uint32_t* to = buf + 52 * t + 12 * j + 2 * half + q;
        to[0] = __byte_perm(p01, p23, 0x5410u);
        to[4] = __byte_perm(p01, p23, 0x7632u);
        to[8] = __byte_perm(h01, h23, 0x5410u);
    }
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
    // byte g / 2 of the four sum words is this shift's
    if (half == 0) {
        const uint32_t u = (static_cast<uint32_t>(sum) + 0x80808080u) ^ 0x80808080u;
#pragma unroll
        for (int d = 0; d < 4; ++d)
            reinterpret_cast<uint8_t*>(buf + 52 * t + 48 + d)[j] = static_cast<uint8_t>(u >> (8 * d));
    }
}

// Block `block` of a token: its integers in registers, and the value of their unit in
// `undo`.  True if the block is wide: the rest is then in `buf`.
template <typename T>
__device__ __forceinline__ bool load_x_bytes(const T* x, int block, int lane, uint32_t* buf, XBytes& o,
                                             float& undo) {
    const int g = lane >> 2, t = lane & 3, j = g >> 1, half = g & 1;
    const T* p = x + 256 * block + 128 * (t >> 1) + 32 * j + 16 * (t & 1) + 8 * half;
    float v[8];
    if constexpr (sizeof(T) == 4) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p));
        const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(w[e] << 16);
            v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
    }
    // the largest |x|, as bits: those of a NaN are above an infinity's (fmaxf would
    // drop it, and its bits pass for an integer below)
    uint32_t top = 0;
#pragma unroll
    for (int l = 0; l < 8; ++l) top = max(top, __float_as_uint(v[l]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    const int e = max(static_cast<int>(top >> 23) - 127, -100);
    // (e = 128: an infinity or NaN in x makes every sum of the block NaN)
    undo = __uint_as_float(e > 127 ? 0x7FC00000u : static_cast<uint32_t>(127 - 21 + e) << 23);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 21 - e) << 23);
    uint32_t w[8], small = 0;
    float rest[8], none[8];
    split_integers(v, up, w, rest);
    bool left = false;
#pragma unroll
    for (int l = 0; l < 8; ++l) {
        small += v[l] != 0.f && (__float_as_uint(v[l]) & 0x7FFFFFFFu) < static_cast<uint32_t>(127 - 9 + e) << 23;
        left |= rest[l] != 0.f;
    }
    store_digits(w, lane, buf);
    __syncwarp();
    const uint4* from = reinterpret_cast<const uint4*>(buf + 52 * t);
#pragma unroll
    for (int c = 0; c < 13; ++c) {
        const uint4 u = from[c];
        uint32_t* to = c < 12 ? o.x[c / 3][c % 3] : o.s;
        to[0] = u.x, to[1] = u.y, to[2] = u.z, to[3] = u.w;
    }
    const bool wide = __reduce_add_sync(0xFFFFFFFFu, small) > kQK / 4 && __any_sync(0xFFFFFFFFu, left);
    if (wide) {
        split_integers(rest, 1 / kRest, w, none);
        __syncwarp();
        store_digits(w, lane, buf);
        __syncwarp();
    }
    return wide;
}

// c + the four products of a's unsigned bytes with b's signed ones.
__device__ __forceinline__ int dot4_us(uint32_t a, uint32_t b, int c) {
    int d;
    asm("dp4a.u32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// One row's slice of a block times one token, all in integers: codes are masked in
// place (4^j q) and meet sc_j 4^(3 - j), so every product carries 64; a digit's sum
// over a slice is below 2^25.
template <typename X>
__device__ __forceinline__ float slice_product(const RowWords& r, const X& x) {
    int a0 = 0, a1 = 0, a2 = 0;
    const int sc[4] = {static_cast<int>((r.sc << 6) & 0x3C0u), static_cast<int>((r.sc >> 4) & 0xF0u),
                       static_cast<int>((r.sc >> 14) & 0x3Cu), static_cast<int>((r.sc >> 24) & 0xFu)};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        int s0 = 0, s1 = 0, s2 = 0;
        const uint4 x0 = x.quad(j, 0), x1 = x.quad(j, 1), x2 = x.quad(j, 2);
        const uint32_t d0[4] = {x0.x, x0.y, x0.z, x0.w}, d1[4] = {x1.x, x1.y, x1.z, x1.w},
                       d2[4] = {x2.x, x2.y, x2.z, x2.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t q = r.q[i] & (0x03030303u << (2 * j));
            s0 = dot4_us(q, d0[i], s0);
            s1 = dot4_us(q, d1[i], s1);
            s2 = dot4_us(q, d2[i], s2);
        }
        a0 += s0 * sc[j];
        a1 += s1 * sc[j];
        a2 += s2 * sc[j];
    }
    // minima, m in the high nibbles: products carry 16
    const uint32_t m = r.sc & 0xF0F0F0F0u;
    const uint4 s = x.sums();
    const int e0 = dot4_us(m, s.x, 0) + 256 * dot4_us(m, s.y, 0);
    const int e1 = dot4_us(m, s.z, 0) + 256 * dot4_us(m, s.w, 0);
    const float a = fmaf(65536.f, static_cast<float>(a2),
                         fmaf(256.f, static_cast<float>(a1), static_cast<float>(a0)));
    const float e = fmaf(65536.f, static_cast<float>(e1), static_cast<float>(e0));
    return fmaf(f16_bits_to_float(r.dd) * 0x1p-6f, a, f16_bits_to_float(r.dd >> 16) * -0x1p-4f * e);
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
    // streamed tiles
    int depth;            // units in flight
    int parts;            // CTAs of a cluster that divide K
    unsigned int* err;
};

enum class Rows { kGated, kLora };

__device__ __forceinline__ void cp_async_word(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}

template <typename T, int NT>
struct Pass {
    static constexpr int kTokens = NT == 0 ? 1 : NT * (sizeof(T) == 4 ? 4 : 8);
    static constexpr int kSums = NT == 0 ? kUnitRows : 32 * NT * (sizeof(T) == 4 ? 2 : 4);  // of a tile
};

// A warp's sums of two tiles, in fragment order.
template <typename T, int NT>
__device__ __forceinline__ void write_sums(float* mine, int lane, const float (&acc)[2][NT][4]) {
    constexpr int kOut = Pass<T, NT>::kSums;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (sizeof(T) == 4) {  // hi and lo columns of a token
                mine[a * kOut + (2 * n) * 32 + lane] = acc[a][n][0] + acc[a][n][1];
                mine[a * kOut + (2 * n + 1) * 32 + lane] = acc[a][n][2] + acc[a][n][3];
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) mine[a * kOut + (4 * n + c) * 32 + lane] = acc[a][n][c];
            }
        }
}

// Weight k of a row of blocks.
__device__ __forceinline__ float weight_at(const uint8_t* row, int k) {
    const uint8_t* b = row + static_cast<size_t>(k / kQK) * kBlockBytes;
    const int half = (k >> 7) & 1, j = (k >> 5) & 3, seg = (k >> 4) & 1;
    const uint32_t sc = b[8 * half + 2 * j + seg];
    const uint32_t q = (b[16 + 32 * half + 16 * seg + (k & 15)] >> (2 * j)) & 3u;
    const uint32_t dd = ld_u32(b + 80);
    const float dl = f16_bits_to_float(dd) * static_cast<float>(sc & 15u);
    return fmaf(dl, static_cast<float>(q), -(f16_bits_to_float(dd >> 16) * static_cast<float>(sc >> 4)));
}

// Whether a word of x holds an infinity or NaN.
template <typename T>
__device__ __forceinline__ bool special_word(uint32_t w) {
    constexpr uint32_t kExp = 0x7F800000u;
    return (w & kExp) == kExp || (sizeof(T) == 2 && ((w << 16) & kExp) == kExp);
}

// A sum over K that came out not finite, of one token and one row: codes and minima
// are summed apart, and x in parts, so infinities meet as NaN where the formula has
// one.  By the formula the sum is that of the infinities and NaNs of x times their
// weights; with x finite the parts overflowed, and the sum is taken of x 2^-64.
// 14336 x 4096: looking for such sums costs a call 0.2 us at one token, 0.1 at 16 bf16
// and 0.7 at eight f32 ones; a token that has them 0.7 ms.  (In line: as a function of
// its own, called or not, it cost every launch 0.3 us on the host.)
template <typename T>
__device__ __forceinline__ float sum_not_finite(const T* x, const uint8_t* row, int K) {
    constexpr int kStep = 32 / sizeof(T);
    float sum = 0.f;
    bool found = false;
#pragma unroll 1
    for (int k = 0; k < K; k += kStep) {
        const uint4 a = *reinterpret_cast<const uint4*>(x + k), b = *reinterpret_cast<const uint4*>(x + k + kStep / 2);
        if (!(special_word<T>(a.x) || special_word<T>(a.y) || special_word<T>(a.z) || special_word<T>(a.w) ||
              special_word<T>(b.x) || special_word<T>(b.y) || special_word<T>(b.z) || special_word<T>(b.w)))
            continue;
        found = true;
#pragma unroll 1
        for (int e = k; e < k + kStep; ++e) {
            const float v = to_float(x[e]);
            if (special_word<float>(__float_as_uint(v))) sum = fmaf(weight_at(row, e), v, sum);
        }
        if (sum != sum) break;
    }
    if (found) return sum;
#pragma unroll 1
    for (int k = 0; k < K; ++k) sum = fmaf(weight_at(row, k), to_float(x[k]) * 0x1p-64f, sum);
    return sum * 0x1p64f;
}

// Sum o of a unit's two tiles -> results.
template <typename T, int NT, Rows kMode>
__device__ __forceinline__ void finish_row(const T* x, const RowsArgs& p, int o, float (&v)[2], int unit,
                                           int m0) {
    constexpr bool kSplit = sizeof(T) == 4;
    const int f = o >> 5, l = o & 31;
    // fragment f of lane l: its row of the tile and its token
    const int r = NT == 0 ? o : (l >> 2) + 8 * (kSplit ? f & 1 : (f >> 1) & 1);
    const int m = m0 + (NT == 0  ? 0
                        : kSplit ? (f >> 1) * 4 + (l & 3)
                                 : (f >> 2) * 8 + 2 * (l & 3) + (f & 1));
    const int n = unit * p.unit_step + r;
    if (m >= p.M) return;
    if (!(fabsf(v[0]) + fabsf(v[1]) <= 3.402823466e38f)) {
        // (each by itself: a row past N is whatever the slot held before)
#pragma unroll 1
        for (int a = 0; a < 2; ++a) {
            const int na = n + a * p.tile1_row;
            if (fabsf(a ? v[1] : v[0]) <= 3.402823466e38f || na >= p.N) continue;
            const float sum = sum_not_finite(x + static_cast<size_t>(m) * p.K,
                                             (a ? p.w1 : p.w0) + static_cast<size_t>(na) * (p.K / kQK) * kBlockBytes,
                                             p.K);
            v[0] = a ? v[0] : sum;
            v[1] = a ? sum : v[1];
        }
    }
    if (kMode == Rows::kGated) {
        if (n >= p.N) return;
        const size_t at = static_cast<size_t>(m) * p.N + n;
        static_cast<T*>(p.h)[at] = from_float<T>(act_value<!kSplit>(v[0], p.act) * v[1]);
        if (p.gate != nullptr) {
            static_cast<T*>(p.gate)[at] = from_float<T>(v[0]);
            static_cast<T*>(p.up)[at] = from_float<T>(v[1]);
        }
    } else {
        const int id = p.ids[m];
        if (id >= 0 && id < p.n_adapters) {
            // sixteen of the rank at a time, both rows': one trip to memory
            const uint4* br[2];
#pragma unroll
            for (int a = 0; a < 2; ++a)
                br[a] = reinterpret_cast<const uint4*>(
                    p.b + (static_cast<size_t>(id) * p.N + min(n + a * p.tile1_row, p.N - 1)) * p.R);
            const float4* tr = reinterpret_cast<const float4*>(p.t + static_cast<size_t>(m) * p.R);
            for (int c = 0; c < p.R / 8; c += 2) {
                const bool two = c + 1 < p.R / 8;
                uint4 bv[2][2];
                float4 tv[4];
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    bv[a][0] = __ldg(br[a] + c);
                    bv[a][1] = two ? __ldg(br[a] + c + 1) : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    tv[q] = q < 2 || two ? tr[2 * c + q] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int a = 0; a < 2; ++a)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t bw[4] = {bv[a][h].x, bv[a][h].y, bv[a][h].z, bv[a][h].w};
                        const float4 t0 = tv[2 * h], t1 = tv[2 * h + 1];
                        const float tt[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            v[a] = fmaf(__uint_as_float(bw[q] << 16), tt[2 * q], v[a]);
                            v[a] = fmaf(__uint_as_float(bw[q] & 0xFFFF0000u), tt[2 * q + 1], v[a]);
                        }
                    }
            }
        } else if (id != -1) {
            v[0] = v[1] = 0.f;  // an id out of range: a zero row
        }
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int na = n + a * p.tile1_row;
            if (na < p.N) static_cast<T*>(p.y)[static_cast<size_t>(m) * p.N + na] = from_float<T>(v[a]);
        }
    }
}

template <typename T, int NT, int S, Rows kMode>
__global__ void __launch_bounds__(kWarps * 32, 1) rows_kernel(const T* __restrict__ x, RowsArgs p) {
    constexpr bool kSplit = sizeof(T) == 4;
    constexpr int kTokens = Pass<T, NT>::kTokens;       // tokens of a pass
    constexpr int kOut = Pass<T, NT>::kSums;            // sums of one tile
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
                        const uint32_t row = ring + (item % kDepth) * kItemBytes +
                                             84 * ((lane >> 2) & 3) + 448 * (lane >> 4);
                        block_product<T, NT>(read_row(row, lane & 3), read_row(row + 896, lane & 3), xb[s],
                                             acc[a]);
                        ++item;
                    }
                }
                // this warp's sums, in fragment order
                write_sums<T, NT>(red + (static_cast<size_t>(u & 1) * p.kw + kw) * (2 * kOut), lane, acc);
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
                    finish_row<T, NT, kMode>(x, p, o, v, unit, m0);
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            // a next pass reuses both sum buffers from its first unit on
            asm volatile("bar.sync %0, %1;" ::"r"(group), "r"(group_threads) : "memory");
        }
    }
    if (!waited) pdl_wait_prerequisites();
}

// The passes over tokens are a grid's y: of more than it holds, the rest go to
// further launches (of the same kernel: a token's result is the same in each).
constexpr int kMaxPasses = 65535;

// Calls `launch(x, args)` for each run of at most kMaxPasses passes of kTokens.
template <typename T, int kTokens, typename Launch>
cudaError_t launch_passes(const T* x, const RowsArgs& p, Launch&& launch) {
    for (int first = 0; first < p.M; first += kMaxPasses * kTokens) {
        RowsArgs q = p;
        q.M = std::min(p.M - first, kMaxPasses * kTokens);
        const size_t at = static_cast<size_t>(first) * p.N;
        if (p.h != nullptr) q.h = static_cast<T*>(p.h) + at;
        if (p.gate != nullptr) q.gate = static_cast<T*>(p.gate) + at;
        if (p.up != nullptr) q.up = static_cast<T*>(p.up) + at;
        if (p.y != nullptr) q.y = static_cast<T*>(p.y) + at;
        if (p.t != nullptr) q.t = p.t + static_cast<size_t>(first) * p.R;
        if (p.ids != nullptr) q.ids = p.ids + first;
        const cudaError_t e = launch(x + static_cast<size_t>(first) * p.K, q);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T, int NT, int S, Rows kMode>
cudaError_t launch_as(const void* x, RowsArgs& p, int device, int sm_count, cudaStream_t stream) {
    constexpr int kTokens = Pass<T, NT>::kTokens;
    constexpr int kOut = Pass<T, NT>::kSums;
    constexpr int kSmem = kWarps * kDepth * kItemBytes + (kWarps * 2 + kGroupUnits) * 2 * kOut * 4 ;
    static_assert(kSmem <= 232448, "shared memory");
    static std::atomic<bool> attr_done[64] = {};  // (set by any thread; setting twice does no harm)
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[device].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(rows_kernel<T, NT, S, kMode>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        attr_done[device].store(true, std::memory_order_release);
    }
    const int blocks = p.K / kQK;
    p.passes = (blocks + kWarps * S - 1) / (kWarps * S);
    const int per_pass = (blocks + p.passes - 1) / p.passes;
    p.kw = (per_pass + S - 1) / S;
    p.groups = p.passes > 1 ? 1 : kWarps / p.kw;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_passes<T, kTokens>(static_cast<const T*>(x), p, [&](const T* xs, const RowsArgs& q) {
        cfg.gridDim = dim3(std::min(sm_count, (p.units + p.groups - 1) / p.groups),
                           (q.M + kTokens - 1) / kTokens);
        return cudaLaunchKernelEx(&cfg, rows_kernel<T, NT, S, kMode>, xs, q);
    });
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// Two words into another CTA of the cluster, counted by a barrier there.
__device__ __forceinline__ void send_pair(uint32_t addr, uint32_t bar, uint32_t rank, float a, float b) {
    asm volatile(
        "{\n\t.reg .u32 ra, rb;\n\tmapa.shared::cluster.u32 ra, %0, %2;\n\t"
        "mapa.shared::cluster.u32 rb, %1, %2;\n\t"
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [ra], {%3, %4}, [rb];\n\t}"
        ::"r"(addr), "r"(bar), "r"(rank), "f"(a), "f"(b)
        : "memory");
}

// The same product with a block for each warp.  A tile of 16 rows, or of a part of
// each, comes by bulk copies, where 84-byte columns take a word a lane (16 copy
// instructions for 16 rows x 256 weights, which the load unit could not issue at
// more than 3.9 TB/s).  The warps' sums meet as above, but a unit late: a warp
// multiplies unit u, then waits for the others' sums of u - 1 and brings its share
// of them out, and only then writes its sums of u, so that two buffers of sums do
// and no warp waits for the slowest at every unit.  That all have their sums of
// u - 1 also says that the unit's slot is free to be refilled: a warp arrives after
// it has stored sums that every word it read went into, so no read is still on its
// way.
// More than 16 blocks: a cluster's CTAs divide K (in fours of blocks, so that
// copies start at 16 bytes).  Each has a share of a unit's outputs; the others send
// it their sums of those, which it adds in the order of K another unit later.  A
// CTA that sends for unit u has brought out u - 2, so its peers have sent theirs
// for u - 2 and brought out u - 4: four buffers need no other bookkeeping.
// NT = 0: one token, as integers (see XBytes).
template <typename T, int NT, Rows kMode>
__global__ void __launch_bounds__(kWarps * 32, 1) stream_kernel(const T* __restrict__ x, RowsArgs p) {
    constexpr bool kBytes = NT == 0;
    constexpr int kTokens = Pass<T, NT>::kTokens, kOut = Pass<T, NT>::kSums;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const int m0 = blockIdx.y * kTokens;
    const int rank = static_cast<int>(blockIdx.x) % p.parts, first_unit = static_cast<int>(blockIdx.x) / p.parts;
    const int unit_step = static_cast<int>(gridDim.x) / p.parts;
    const int blocks = p.K / kQK;
    const size_t row_bytes = static_cast<size_t>(blocks) * kBlockBytes;
    // this CTA's blocks
    const int b0 = p.parts == 1 ? 0 : 4 * (blocks / 4 * rank / p.parts);
    const int nb = p.parts == 1 ? blocks : 4 * (blocks / 4 * (rank + 1) / p.parts) - b0;
    const int pitch = nb * kBlockBytes, tile_bytes = kUnitRows * pitch;
    const int slot_bytes = 2 * kUnitRows * min(blocks, kWarps) * kBlockBytes;
    float* red = reinterpret_cast<float*>(smem);
    // sums from the cluster's CTAs: [unit % 4][from][output of the share]
    const int share = kOut / p.parts + 1;
    float2* inbox = reinterpret_cast<float2*>(red + kWarps * 2 * 2 * kOut);
    uint32_t* xs = reinterpret_cast<uint32_t*>(inbox + 4 * (kOut + kMaxRowParts));
    uint8_t* slots = reinterpret_cast<uint8_t*>(xs + (kBytes ? kWarps * kXWords : 0));
    const uint32_t bars = smem_u32(slots + static_cast<size_t>(p.depth) * slot_bytes);
    const uint32_t bar_sums = bars + 8 * kMaxDepth, bar_inbox = bar_sums + 8;
    volatile int* abort_flag =
        reinterpret_cast<volatile int*>(slots + static_cast<size_t>(p.depth) * slot_bytes + 8 * (kMaxDepth + 5));
    const int my_units = (p.units - 1 - first_unit) / unit_step + 1;
    // by a whole warp
    auto issue = [&](int u) {
        if (u >= my_units) return;
        const int unit = first_unit + u * unit_step;
        uint8_t* slot = slots + static_cast<size_t>(u % p.depth) * slot_bytes;
        const uint32_t bar = bars + 8 * (u % p.depth);
        const int tile = lane >> 4;
        const int row0 = unit * p.unit_step + (tile ? p.tile1_row : 0);
        const int valid = min(max(p.N - row0, 0), kUnitRows);
        const uint8_t* src = (tile ? p.w1 : p.w0) + static_cast<size_t>(row0) * row_bytes;
        uint8_t* dst = slot + tile * tile_bytes;
        uint32_t bytes = static_cast<uint32_t>(valid * pitch);
        if (p.parts == 1) {
            // one copy a tile (the matrix may end off 16 bytes)
            if ((lane & 15) == 0)
                for (uint32_t at = bytes & ~15u; at < bytes; at += 4)
                    *reinterpret_cast<uint32_t*>(dst + at) = __ldg(reinterpret_cast<const uint32_t*>(src + at));
            bytes &= ~15u;
        }
        const uint32_t other = __shfl_sync(0xFFFFFFFFu, bytes, 16);
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes + other);
        __syncwarp();
        if (p.parts == 1) {
            if ((lane & 15) == 0 && bytes != 0) bulk_copy_g2s(smem_u32(dst), src, bytes, bar);
        } else if ((lane & 15) < valid) {
            bulk_copy_g2s(smem_u32(dst + (lane & 15) * pitch),
                          src + (lane & 15) * row_bytes + static_cast<size_t>(b0) * kBlockBytes, pitch, bar);
        }
    };
    pdl_allow_dependents();
    bool waited = false;
    if (warp == 0) {
        if (lane == 0) {
            *abort_flag = 0;
            for (int d = 0; d < p.depth; ++d) mbar_init(bars + 8 * d, 1);
            mbar_init(bar_sums, kWarps);
            for (int d = 0; d < 4; ++d) mbar_init(bar_inbox + 8 * d, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        if (!p.const_weights) {
            pdl_wait_prerequisites();
            waited = true;
        }
        for (int d = 0; d < p.depth; ++d) issue(d);
    }
    if (!waited && !p.x_ready) {
        pdl_wait_prerequisites();
        waited = true;
    }
    XBytes xi;
    [[maybe_unused]] float undo = 0.f;
    [[maybe_unused]] bool wide = false;
    XBlock<T> xm[kBytes ? 1 : NT];
    if (warp < nb) {
        if constexpr (kBytes) {
            wide = load_x_bytes(x, b0 + warp, lane, xs + warp * kXWords, xi, undo);
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n)
                load_x_block(x, p.K, b0 + warp, m0 + n * (kTokens / NT), p.M, lane, xm[n]);
        }
    }
    const int o_first = kOut * rank / p.parts, o_count = kOut * (rank + 1) / p.parts - o_first;
    // the warps take turns at the outputs of a unit, and at refilling its slot
    auto turn_at = [&](int u) { return (warp + u) & (kWarps - 1); };
    // unit u: the warps' sums -> results, or to the CTAs that have them
    auto bring_out = [&](int u) {
        mbar_wait_bounded(bar_sums, u & 1, abort_flag, p.err, kErrTimeoutAccum);
        if (turn_at(u) == kWarps - 1) issue(u + p.depth);
        if (kMode == Rows::kLora && !waited) {
            pdl_wait_prerequisites();  // t
            waited = true;
        }
        const float* all = red + (u & 1) * kWarps * (2 * kOut);
        for (int o = 32 * turn_at(u) + lane; o < kOut; o += 32 * kWarps) {
            float v[2] = {0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                v[0] += all[w * (2 * kOut) + o];
                v[1] += all[w * (2 * kOut) + kOut + o];
            }
            if (p.parts == 1) {
                finish_row<T, NT, kMode>(x, p, o, v, first_unit + u * unit_step, m0);
            } else {
                const int to = ((o + 1) * p.parts - 1) / kOut;  // whose share o is
                const int at = ((u & 3) * p.parts + rank) * share + o - kOut * to / p.parts;
                send_pair(smem_u32(inbox + at), bar_inbox + 8 * (u & 3), to, v[0], v[1]);
            }
        }
    };
    // unit u: the cluster's sums -> results
    auto finish_parts = [&](int u) {
        if (turn_at(u) == kWarps - 1 && lane == 0)
            mbar_arrive_expect_tx(bar_inbox + 8 * (u & 3), 8 * p.parts * o_count);
        if (32 * turn_at(u) >= o_count) return;
        tc::wait_peer_bounded(bar_inbox + 8 * (u & 3), (u >> 2) & 1, abort_flag, p.err, kErrTimeoutFull);
        for (int o = 32 * turn_at(u) + lane; o < o_count; o += 32 * kWarps) {
            float v[2] = {0.f, 0.f};
            for (int z = 0; z < p.parts; ++z) {
                const float2 w = inbox[((u & 3) * p.parts + z) * share + o];
                v[0] += w.x;
                v[1] += w.y;
            }
            finish_row<T, NT, kMode>(x, p, o_first + o, v, first_unit + u * unit_step, m0);
        }
    };
    __syncthreads();
    if (p.parts > 1) {  // every CTA's barriers are there before anything is sent
        cluster_arrive();
        cluster_wait();
    }
    for (int u = 0; u < my_units; ++u) {
        const uint32_t slot = smem_u32(slots) + (u % p.depth) * slot_bytes;
        mbar_wait_bounded(bars + 8 * (u % p.depth), (u / p.depth) & 1, abort_flag, p.err, kErrTimeoutFull);
        float* mine = red + ((u & 1) * kWarps + warp) * (2 * kOut);
        const uint32_t row = slot + warp * kBlockBytes + (lane >> 2) * pitch;
        // (one token: rows lane / 4 and 8 on of the two tiles)
        float acc[2][kBytes ? 1 : NT][4] = {};
        if (warp < nb) {
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const RowWords r0 = read_row(row + a * tile_bytes, lane & 3);
                const RowWords r1 = read_row(row + a * tile_bytes + 8 * pitch, lane & 3);
                if constexpr (kBytes) {
                    acc[a][0][0] = undo * slice_product(r0, xi);
                    acc[a][0][1] = undo * slice_product(r1, xi);
                } else {
                    block_product<T, NT>(r0, r1, xm, acc[a]);
                }
            }
            if constexpr (kBytes) {
                if (wide) {  // (of the warp)
                    const StoredXBytes rest = {
                        reinterpret_cast<const uint4*>(xs + warp * kXWords + 52 * (lane & 3))};
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        const RowWords r = read_row(row + (i >> 1) * tile_bytes + (i & 1) * 8 * pitch, lane & 3);
                        const float v = undo * kRest * slice_product(r, rest);
#pragma unroll
                        for (int o = 0; o < 4; ++o) acc[o >> 1][0][o & 1] += i == o ? v : 0.f;
                    }
                }
            }
        }
        if (u > 0) bring_out(u - 1);
        if (p.parts > 1 && u > 1) finish_parts(u - 2);
        if constexpr (kBytes) {
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float v = acc[a][0][r];
                    v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
                    v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
                    if ((lane & 3) == 0) mine[a * kOut + 8 * r + (lane >> 2)] = v;
                }
        } else {
            write_sums<T, NT>(mine, lane, acc);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_sums);
    }
    bring_out(my_units - 1);
    if (p.parts > 1) {
        if (my_units > 1) finish_parts(my_units - 2);
        finish_parts(my_units - 1);
        cluster_arrive();  // no CTA leaves while another may send to it
        cluster_wait();
    }
    if (!waited) pdl_wait_prerequisites();
    if (*abort_flag) {
        // no copy may still write shared memory when it is given back
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {}
    }
}

// Whether the product can be streamed, and how.
template <typename T, int NT>
bool plan_stream(RowsArgs& p, size_t& smem) {
    const int blocks = p.K / kQK;
    if (blocks <= kWarps / 2) return false;
    if (((reinterpret_cast<uintptr_t>(p.w0) | reinterpret_cast<uintptr_t>(p.w1)) & 15) != 0) return false;
    p.parts = (blocks + kWarps - 1) / kWarps;
    if (p.parts > 1 && (p.parts > kMaxRowParts || blocks % 4 != 0)) return false;
    const size_t fixed = kWarps * 2 * 2 * Pass<T, NT>::kSums * 4 + 4 * (Pass<T, NT>::kSums + kMaxRowParts) * 8 +
                         (NT == 0 ? static_cast<size_t>(kWarps) * kXWords * 4 : 0) + 8 * (kMaxDepth + 5) + 16;
    const size_t unit = 2 * static_cast<size_t>(kUnitRows) * std::min(blocks, kWarps) * kBlockBytes;
    p.depth = static_cast<int>(std::min<size_t>(kMaxDepth, (kMaxSmem - fixed) / unit));
    smem = fixed + p.depth * unit;
    return true;
}

template <typename T, int NT, Rows kMode>
cudaError_t launch_stream(const void* x, RowsArgs& p, size_t smem, int device, int sm_count,
                          cudaStream_t stream) {
    // clusters of a size that the GPU holds at once, 0: not known yet
    static std::atomic<int> resident[64][kMaxRowParts + 1] = {};
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    cudaError_t e = ffn_error_word(device, &p.err);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.parts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.parts > 1 ? 2 : 1;
    int most = resident[device][p.parts].load(std::memory_order_acquire);
    if (most == 0) {
        e = cudaFuncSetAttribute(stream_kernel<T, NT, kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kMaxSmem);
        if (e != cudaSuccess) return e;
        most = sm_count;
        if (p.parts > 1) {
            cfg.gridDim = dim3(sm_count / p.parts * p.parts);
            e = cudaOccupancyMaxActiveClusters(&most, stream_kernel<T, NT, kMode>, &cfg);
            if (e != cudaSuccess) return e;
        }
        most = std::max(1, most);
        resident[device][p.parts].store(most, std::memory_order_release);
    }
    constexpr int kTokens = Pass<T, NT>::kTokens;
    return launch_passes<T, kTokens>(static_cast<const T*>(x), p, [&](const T* xs, const RowsArgs& q) {
        cfg.gridDim = dim3(std::min(most, p.units) * p.parts, (q.M + kTokens - 1) / kTokens);
        return cudaLaunchKernelEx(&cfg, stream_kernel<T, NT, kMode>, xs, q);
    });
}

// Columns of x in registers: one tile of eight and up to two blocks a warp, or
// two tiles (more than 8 bf16 or 4 f32 tokens) and one block.
template <typename T, Rows kMode>
cudaError_t launch_rows_mode(const void* x, RowsArgs& p, int device, int sm_count,
                             cudaStream_t stream) {
    constexpr int kOne = sizeof(T) == 4 ? 4 : 8;
    size_t smem = 0;
    if (p.M == 1 && plan_stream<T, 0>(p, smem))
        return launch_stream<T, 0, kMode>(x, p, smem, device, sm_count, stream);
    if (p.M <= kOne && plan_stream<T, 1>(p, smem))
        return launch_stream<T, 1, kMode>(x, p, smem, device, sm_count, stream);
    if (p.M > kOne && plan_stream<T, 2>(p, smem))
        return launch_stream<T, 2, kMode>(x, p, smem, device, sm_count, stream);
    if (p.M > kOne)
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
