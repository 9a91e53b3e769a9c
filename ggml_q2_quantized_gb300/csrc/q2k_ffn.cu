// Feed-forward operators on Q2_K weights: the gated block, its backward pass
// and a projection with one low-rank adapter per token.
//
//   gated     g = x Wg^T, u = x Wu^T, h = act(g) * u
//   backward  dg = dh u act'(g), du = dh act(g), dx = dg Wg + du Wu
//   lora      y_i = W x_i + s_a B_a (A_a x_i), a the adapter of token i
//
// Every weight is formed in f32 (dl q - ml rounded once) and every sum is f32.
#include <cuda_runtime.h>

#include <algorithm>

#include "q2k_device.cuh"
#include "q2k_ffn.cuh"
#include "q2k_internal.h"

namespace q2k {

namespace {

// ---- t = s_a A_a x ---------------------------------------------------------------
//
// One cluster of eight CTAs takes 16 of an adapter's rows and the tokens with
// that adapter among eight or 32 consecutive ones: A_a's rows are the MMA's rows,
// eight tokens its columns, and the cluster's 64 warps divide K, so that even one
// token's A_a (128 KB at rank 16, K = 4096) is read by eight SMs at once.  Sums
// meet in shared memory, then over the cluster, in a fixed order.  A token takes
// only its own adapter's column.  An f32 x is three bf16 parts (24 bits).  The
// time is the latency of a few dependent loads: a warp asks for four of its
// K-steps at once.
constexpr int kShrinkWarps = 8;
constexpr int kShrinkCtas = 8;
constexpr int kShrinkRows = 16;
// Up to this many tokens a cluster is launched per token, and the first token
// with an adapter among its eight does the work: eight tokens with eight
// adapters then run at once.  Above, a cluster takes 32 tokens and loops over
// their adapters, which reads A_a a quarter as often (prompts of one adapter).
constexpr int kShrinkPerToken = 64;

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The parts of eight consecutive x as B fragments of two K-steps.
template <typename T>
struct XParts;
template <>
struct XParts<__nv_bfloat16> {
    static constexpr int kParts = 1;
    uint32_t v[1][4];
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
        v[0][0] = a.x, v[0][1] = a.y, v[0][2] = a.z, v[0][3] = a.w;
    }
    __device__ __forceinline__ void zero() { v[0][0] = v[0][1] = v[0][2] = v[0][3] = 0u; }
};
template <>
struct XParts<float> {
    static constexpr int kParts = 3;
    uint32_t v[3][4];
    __device__ __forceinline__ void load(const float* p) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p));
        const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
                v[q][e] = *reinterpret_cast<const uint32_t*>(&h);
                f[2 * e] -= __uint_as_float(v[q][e] << 16);
                f[2 * e + 1] -= __uint_as_float(v[q][e] & 0xFFFF0000u);
                // (an infinity is its first part alone: the others would be NaN, and are 2^120)
                if (q > 0) v[q][e] = min_bf16x2(v[q][e], 0x7B807B80u);
            }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int q = 0; q < 3; ++q) v[q][0] = v[q][1] = v[q][2] = v[q][3] = 0u;
    }
};

// kGroups: groups of eight tokens per cluster (1: launched per token); kSplit:
// clusters that divide the adapters of those tokens.
template <typename T, int kGroups, int kSplit>
__global__ void __cluster_dims__(1, 1, kShrinkCtas) __launch_bounds__(kShrinkWarps * 32)
lora_shrink_kernel(const T* __restrict__ x, const __nv_bfloat16* __restrict__ a,
                   const float* __restrict__ scales, const int* __restrict__ ids,
                   float* __restrict__ t, unsigned int* __restrict__ bad_ids, int M, int K, int R,
                   int n_adapters, unsigned int* __restrict__ counts, int n_counts) {
    constexpr int kSums = kGroups * 4 * 32;  // of a warp: groups x fragment x lanes
    __shared__ float red[kShrinkWarps][kSums];
    __shared__ float part[kSums];
    pdl_allow_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.z;  // = the rank in the cluster
    if (blockIdx.x == 0 && blockIdx.y == 0 && rank == kShrinkCtas - 1) {
        int bad = 0;
        for (int c0 = 0; c0 < M; c0 += kShrinkWarps * 32) {
            const int id = c0 + tid < M ? ids[c0 + tid] : -1;
            bad += __syncthreads_count(id < -1 || id >= n_adapters);
        }
        if (tid == 0) *bad_ids = static_cast<unsigned>(bad);
        for (int c = tid; c < n_counts; c += kShrinkWarps * 32) counts[c] = 0u;
    }
    const int g = lane >> 2, q4 = lane & 3;
    const int block = static_cast<int>(blockIdx.x) / kSplit;
    int skip = static_cast<int>(blockIdx.x) % kSplit;  // until this cluster's next adapter
    const int m0 = kGroups == 1 ? block & ~7 : 8 * kGroups * block;
    const int r0 = blockIdx.y * kShrinkRows;
    int id[kGroups];  // of this lane's column in each group; -1 once done
#pragma unroll
    for (int n = 0; n < kGroups; ++n) {
        const int m = m0 + 8 * n + g;
        id[n] = m < M ? ids[m] : -1;
        if (id[n] >= n_adapters || id[n] < 0) id[n] = -1;
    }
    while (true) {
        // the first adapter left, and its first token
        int ad = -1, token = 0;
#pragma unroll
        for (int n = 0; n < kGroups; ++n) {
            const unsigned has = __ballot_sync(0xFFFFFFFFu, id[n] >= 0);
            if (has != 0 && ad < 0) {
                const int l = __ffs(has) - 1;  // (lane 4 c holds token c's id)
                ad = __shfl_sync(0xFFFFFFFFu, id[n], l);
                token = m0 + 8 * n + (l >> 2);
            }
        }
        if (ad < 0) break;
        bool mine[kGroups];
#pragma unroll
        for (int n = 0; n < kGroups; ++n) {
            mine[n] = id[n] == ad;
            if (mine[n]) id[n] = -1;
        }
        if (kGroups == 1 && token != block) continue;
        if (kSplit > 1) {
            if (skip-- > 0) continue;
            skip = kSplit - 1;
        }
        float acc[kGroups][4] = {};
        const bool ok0 = r0 + g < R, ok1 = r0 + g + 8 < R;
        const __nv_bfloat16* arow = a + (static_cast<size_t>(ad) * R + r0 + g) * K + 8 * q4;
        const T* xrow[kGroups];
#pragma unroll
        for (int n = 0; n < kGroups; ++n)
            xrow[n] = x + static_cast<size_t>(mine[n] ? m0 + 8 * n + g : 0) * K + 8 * q4;
        constexpr int kStep = 32 * kShrinkWarps * kShrinkCtas;
        constexpr int kAhead = kGroups == 1 ? 4 : 2;
        for (int k0 = 32 * (rank * kShrinkWarps + warp); k0 < K; k0 += kAhead * kStep) {
            uint4 lo[kAhead], hi[kAhead];
            XParts<T> xp[kAhead][kGroups];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int k = k0 + u * kStep;
                lo[u] = hi[u] = make_uint4(0u, 0u, 0u, 0u);
                if (k < K && ok0) lo[u] = __ldg(reinterpret_cast<const uint4*>(arow + k));
                if (k < K && ok1)
                    hi[u] = __ldg(reinterpret_cast<const uint4*>(arow + static_cast<size_t>(8) * K + k));
#pragma unroll
                for (int n = 0; n < kGroups; ++n) {
                    if (k < K && mine[n]) xp[u][n].load(xrow[n] + k);
                    else xp[u][n].zero();
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
#pragma unroll
                for (int n = 0; n < kGroups; ++n)
#pragma unroll
                    for (int p = XParts<T>::kParts - 1; p >= 0; --p) {
                        const auto& v = xp[u][n].v[p];
                        mma_bf16_16816(acc[n], lo[u].x, hi[u].x, lo[u].y, hi[u].y, v[0], v[1]);
                        mma_bf16_16816(acc[n], lo[u].z, hi[u].z, lo[u].w, hi[u].w, v[2], v[3]);
                    }
        }
#pragma unroll
        for (int n = 0; n < kGroups; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) red[warp][(4 * n + c) * 32 + lane] = acc[n][c];
        __syncthreads();
        for (int i = tid; i < kSums; i += kShrinkWarps * 32) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kShrinkWarps; ++w) v += red[w][i];
            part[i] = v;
        }
        cluster_sync();
        // each CTA of the cluster adds an eighth of the values over the CTAs
        constexpr int kEach = kSums / kShrinkCtas;
        if (tid < kEach) {
            const int i = rank * kEach + tid;
            const uint32_t at = smem_u32(part + i);
            float v[kShrinkCtas];
#pragma unroll
            for (int c = 0; c < kShrinkCtas; ++c)
                asm volatile(
                    "{\n\t.reg .u32 ra;\n\tmapa.shared::cluster.u32 ra, %1, %2;\n\t"
                    "ld.shared::cluster.f32 %0, [ra];\n\t}"
                    : "=f"(v[c])
                    : "r"(at), "r"(c)
                    : "memory");
#pragma unroll
            for (int c = 1; c < kShrinkCtas; ++c) v[0] += v[c];
            // value f of lane l: row l / 4 + 8 (f / 2 % 2), column 2 (l % 4) + f % 2
            // of group f / 4
            const int f = i >> 5, l = i & 31;
            const int r = r0 + (l >> 2) + 8 * ((f >> 1) & 1);
            const int col = m0 + 8 * (f >> 2) + 2 * (l & 3) + (f & 1);
            if (r < R && col < M && ids[col] == ad)
                t[static_cast<size_t>(col) * R + r] = scales != nullptr ? v[0] * scales[ad] : v[0];
        }
        cluster_sync();  // the values are read before any CTA leaves or goes on
    }
}

template <typename T>
cudaError_t launch_shrink(const LoraArgs& a, float* t, unsigned int* counts, int n_counts,
                          cudaStream_t stream) {
    const T* x = static_cast<const T*>(a.x);
    const unsigned rows = (a.R + kShrinkRows - 1) / kShrinkRows;
    if (a.M <= kShrinkPerToken)
        lora_shrink_kernel<T, 1, 1><<<dim3(a.M, rows, kShrinkCtas), kShrinkWarps * 32, 0, stream>>>(
            x, a.a, a.scales, a.ids, t, a.bad_ids, a.M, a.K, a.R, a.n_adapters, counts, n_counts);
    else {
        // windows of 32 tokens; f32 takes 16, its three parts of x more registers
        // (512 tokens, 7168 x 7168, rank 64: 118 us with 32, 98 with 16).  Two
        // clusters share a window's adapters while all run at once (256 tokens of 16
        // adapters in any order, 7168 wide: 95 us with one and 79 with two; many
        // tokens' empty clusters cost: 2048, rank 128, 446 and 453).
        constexpr int kGroups = sizeof(T) == 4 ? 2 : 4;
        const unsigned windows = (a.M + 8 * kGroups - 1) / (8 * kGroups);
        if (windows * rows * kShrinkCtas <= static_cast<unsigned>(a.sm_count))
            lora_shrink_kernel<T, kGroups, 2>
                <<<dim3(2 * windows, rows, kShrinkCtas), kShrinkWarps * 32, 0, stream>>>(
                    x, a.a, a.scales, a.ids, t, a.bad_ids, a.M, a.K, a.R, a.n_adapters, counts, n_counts);
        else
            lora_shrink_kernel<T, kGroups, 1>
                <<<dim3(windows, rows, kShrinkCtas), kShrinkWarps * 32, 0, stream>>>(
                    x, a.a, a.scales, a.ids, t, a.bad_ids, a.M, a.K, a.R, a.n_adapters, counts, n_counts);
    }
    return cudaGetLastError();
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

bool ffn_rows_path(int m, bool bf16) { return m <= (bf16 ? 16 : 8); }

size_t gated_workspace_bytes(const GatedArgs& a) {
    return a.tensor ? gated_tc_workspace_bytes(a) : 0;
}

cudaError_t launch_gated(const GatedArgs& a, void* workspace, cudaStream_t stream) {
    return a.tensor ? launch_gated_tc(a, workspace, stream) : launch_gated_rows(a, stream);
}

// Workspace: t, then the tensor path's.
static size_t lora_t_bytes(const LoraArgs& a) { return align256(static_cast<size_t>(a.M) * a.R * 4); }

size_t lora_workspace_bytes(const LoraArgs& a) {
    return lora_t_bytes(a) + (a.tensor ? lora_tc_workspace_bytes(a) : 0);
}

cudaError_t launch_lora(const LoraArgs& a, void* workspace, cudaStream_t stream) {
    float* t = static_cast<float*>(workspace);
    uint8_t* rest = static_cast<uint8_t*>(workspace) + lora_t_bytes(a);
    unsigned int* counts = nullptr;
    int n_counts = 0;
    if (a.tensor) lora_tc_counts(a, rest, &counts, &n_counts);
    const cudaError_t e = a.bf16 ? launch_shrink<__nv_bfloat16>(a, t, counts, n_counts, stream)
                                 : launch_shrink<float>(a, t, counts, n_counts, stream);
    if (e != cudaSuccess) return e;
    if (!a.tensor) return launch_lora_rows(a, t, stream);
    return launch_lora_tc(a, t, rest, stream);
}

}  // namespace q2k
