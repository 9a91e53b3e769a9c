// tcgen05, tensor memory, TMA and cluster wrappers of the feed-forward
// operators' tensor-core kernels (sm_103a), and the pieces of the Q2_K decode
// that those kernels share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "q2k_device.cuh"

namespace q2k {
namespace tc {

constexpr int kRows = 128;             // rows of a CTA's tile = TMEM lanes
constexpr int kStageK = 64;            // K elements per stage: one 128-byte swizzle row
constexpr int kBoxBytes = 112;         // bytes per row of a raw-weight TMA box
// bf16 tile image of a [rows, K] matrix: super-tiles of 256 rows x 64 K (32 KB,
// 128-byte swizzled, K-major), super-tile (t, stage s) at (t * stages + s) * 32 KB.
constexpr int kSuperRows = 256;
constexpr int kSuperBytes = kSuperRows * kStageK * 2;

__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Tensor memory, MMAs and commits come in two forms: of one CTA, or (kDuo) of a
// pair of CTAs whose cluster ranks differ in the lowest bit (cta_group::2).
template <bool kDuo>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
    if constexpr (kDuo) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}
template <bool kDuo>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
    if constexpr (kDuo)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols)
                     : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols)
                     : "memory");
}

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups
// 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) |
           (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// The same for an operand stored with its rows (M) running: 64 rows are 128
// contiguous bytes, eight K steps of those 1024 bytes (swizzled as above), the
// next eight K right behind, the next 64 rows `mn_step` bytes further.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr, uint32_t mn_step) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (uint64_t(mn_step >> 4) << 16) |
           (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
constexpr uint32_t kIdescAMnMajor = 1u << 15;
// Instruction descriptor, kind::f16: D f32, A and B bf16, both K-major.
__device__ __forceinline__ uint32_t bf16_idesc(int m, int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}
// D[tmem_d] (+)= A * B^T, both in shared memory.  A pair's MMA takes its rows, and
// half of its columns' B, from the same places of both CTAs.
template <bool kDuo>
__device__ __forceinline__ void mma(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                    uint32_t accumulate) {
    if constexpr (kDuo)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
}
// The same for one CTA with A in tensor memory.
__device__ __forceinline__ void mma_tmem_a(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                           uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(tmem_d), "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// True in one lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Arrive at `bar` (of a pair: in both CTAs) when this thread's MMAs are done.
template <bool kDuo>
__device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (kDuo) {
        const uint16_t both = static_cast<uint16_t>(3u << (cluster_rank() & ~1u));
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
            "[%0], %1;" ::"r"(bar), "h"(both)
            : "memory");
    } else {
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
            : "memory");
    }
}
// As mbar_wait_bounded, for a barrier that another CTA of the cluster arrives at.
__device__ __forceinline__ bool wait_peer_bounded(uint32_t bar, uint32_t parity, volatile int* abort,
                                                  unsigned int* err, uint32_t err_bit) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 1000;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if (it == 1) t0 = global_timer_ns();
        if ((it & 7u) == 0u) {
            if (*abort) return false;
            if (global_timer_ns() - t0 > 1000000000ull) {
                atomicOr(err, err_bit);
                *abort = 1;
                return false;
            }
        }
    }
}
// Arrive at the first CTA's barrier at this CTA's address `bar`.
__device__ __forceinline__ void arrive_first_of_pair(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .u32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [ra];\n\t}"
        ::"r"(bar), "r"(cluster_rank() & ~1u)
        : "memory");
}
// Eight consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_store8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
          "r"(v[6]), "r"(v[7])
        : "memory");
}
__device__ __forceinline__ void tmem_store_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Sixteen consecutive columns (f32) of this thread's TMEM lane.
__device__ __forceinline__ void tmem_load16(uint32_t taddr, float (&f)[16]) {
    uint32_t v[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int q = 0; q < 16; ++q) f[q] = __uint_as_float(v[q]);
}

// 2-D tiled TMA load of the box at (x, y) into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// The same of a 3-D map.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// 4-byte asynchronous copy; src_bytes 0 writes a zero word.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(src_bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Give bulk copies that may still be in flight after a time-out 50 us to land.
__device__ __forceinline__ void linger() {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 50000ull) __nanosleep(1000);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// Byte offset of 16-byte chunk `c` (8 K-elements) of row `r` in a swizzled tile.
__device__ __forceinline__ uint32_t sw128_offset(int r, int c) {
    return static_cast<uint32_t>((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}
// Byte address of chunk `c` (K / 8 of them) of row `m` in a tile image.
__device__ __forceinline__ size_t image_offset(int m, int c, int stages) {
    return (static_cast<size_t>(m / kSuperRows) * stages + (c >> 3)) * kSuperBytes +
           sw128_offset(m % kSuperRows, c & 7);
}

// The four bf16 weights {-ml, dl - ml, 2 dl - ml, 3 dl - ml} of a scale byte,
// each formed in f32 (one rounding) and then rounded to bf16 for the MMA.
__device__ __forceinline__ void weight_table(uint32_t sc, float d, float dmin, uint32_t& lo,
                                             uint32_t& hi) {
    const float dl = __fmul_rn(d, static_cast<float>(sc & 15u));
    const float ml = __fmul_rn(dmin, static_cast<float>(sc >> 4));
    lo = pack_bf16(-ml, __fsub_rn(dl, ml));
    hi = pack_bf16(fmaf(2.f, dl, -ml), fmaf(3.f, dl, -ml));
}
// Byte permute selectors of the four codes of a quant word at shift 2 J: byte i
// becomes the nibbles (2 q_i, 2 q_i + 1) that pick table entry q_i.
template <int J>
__device__ __forceinline__ uint32_t code_selectors(uint32_t word) {
    const uint32_t t2 = (J == 0 ? word * 2u : word >> (2 * J - (J > 0))) & 0x06060606u;
    return t2 * 0x11u + 0x10101010u;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (null when
// the driver has none).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();
// Raw Q2_K weights as a 2-D byte tensor (N rows of K/256 * 84 bytes) with a box
// of `rows` rows x 112 bytes; false unless rows are multiples of 16 bytes (K a
// multiple of 1024) and the base is 16-byte aligned.
// (of `group` rows together as one of the map's; false if those do not start at 16 bytes)
// matrices > 0: that many such matrices, one after another, as a 3-D tensor with boxes
// of one.
bool make_weight_map(CUtensorMap* map, const uint8_t* w, int N, int K, int rows, int group, int matrices);

}  // namespace tc
}  // namespace q2k
