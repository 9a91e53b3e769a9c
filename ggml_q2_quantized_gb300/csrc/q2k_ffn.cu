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

constexpr int kTok = 8;  // tokens per pass over a weight row

// Weight `i` (0..255) of the block at `blk`.
__device__ __forceinline__ float block_weight(const uint8_t* blk, int i) {
    const int h = i >> 7, j = (i >> 5) & 3, seg = (i >> 4) & 1, l = i & 15;
    const uint32_t sc = blk[8 * h + 2 * j + seg];
    const uint32_t q = (blk[16 + 32 * h + 16 * seg + l] >> (2 * j)) & 3u;
    const uint32_t dd = ld_u32(blk + 80);
    const float dl = f16_bits_to_float(dd) * static_cast<float>(sc & 15u);
    const float ml = f16_bits_to_float(dd >> 16) * static_cast<float>(sc >> 4);
    return fmaf(dl, static_cast<float>(q), -ml);
}

// One warp: the dot products of weight row `row` with tokens m0 .. m0 + count - 1.
template <typename T>
__device__ __forceinline__ void row_dots(const T* x, const uint8_t* row, int K, int m0, int count,
                                         float (&acc)[kTok]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int t = 0; t < kTok; ++t) acc[t] = 0.f;
    for (int b = 0; b < K / kQK; ++b)
        for (int i = lane; i < kQK; i += 32) {
            const float w = block_weight(row + static_cast<size_t>(b) * kBlockBytes, i);
            for (int t = 0; t < count; ++t)
                acc[t] = fmaf(w, to_float(x[static_cast<size_t>(m0 + t) * K + b * kQK + i]), acc[t]);
        }
    for (int t = 0; t < count; ++t)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xFFFFFFFFu, acc[t], o);
}

template <typename T>
__global__ void __launch_bounds__(256)
gated_rows_kernel(const T* __restrict__ x, const uint8_t* __restrict__ wg,
                  const uint8_t* __restrict__ wu, T* __restrict__ h, T* __restrict__ gate,
                  T* __restrict__ up, int M, int N, int K, int act) {
    const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (n >= N) return;
    const size_t off = static_cast<size_t>(n) * (K / kQK) * kBlockBytes;
    for (int m0 = 0; m0 < M; m0 += kTok) {
        const int count = min(kTok, M - m0);
        float g[kTok], u[kTok];
        row_dots(x, wg + off, K, m0, count, g);
        row_dots(x, wu + off, K, m0, count, u);
        if ((threadIdx.x & 31) == 0)
            for (int t = 0; t < count; ++t) {
                const size_t o = static_cast<size_t>(m0 + t) * N + n;
                h[o] = from_float<T>(act_value(g[t], act) * u[t]);
                if (gate != nullptr) {
                    gate[o] = from_float<T>(g[t]);
                    up[o] = from_float<T>(u[t]);
                }
            }
    }
}

// dg, du (f32, [m, n] each) and their copies for the caller.
__global__ void __launch_bounds__(256)
gated_grad_kernel(const __nv_bfloat16* __restrict__ dh, const __nv_bfloat16* __restrict__ gate,
                  const __nv_bfloat16* __restrict__ up, float* __restrict__ dg,
                  float* __restrict__ du, __nv_bfloat16* __restrict__ dgate,
                  __nv_bfloat16* __restrict__ dup, size_t count, int act) {
    for (size_t i = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < count;
         i += static_cast<size_t>(gridDim.x) * blockDim.x) {
        float v, s;
        act_value_slope(to_float(gate[i]), act, v, s);
        const float d = to_float(dh[i]);
        dg[i] = d * to_float(up[i]) * s;
        du[i] = d * v;
        if (dgate != nullptr) {
            dgate[i] = from_float<__nv_bfloat16>(dg[i]);
            dup[i] = from_float<__nv_bfloat16>(du[i]);
        }
    }
}

// dx[m0.., k] for one column k per thread: a sum over the rows of Wg and Wu.
__global__ void __launch_bounds__(128)
gated_dx_kernel(const float* __restrict__ dg, const float* __restrict__ du,
                const uint8_t* __restrict__ wg, const uint8_t* __restrict__ wu,
                __nv_bfloat16* __restrict__ dx, int M, int N, int K) {
    const int k = blockIdx.x * blockDim.x + threadIdx.x;  // K is a multiple of 128
    const int m0 = blockIdx.y * kTok;
    const int count = min(kTok, M - m0);
    const size_t row_bytes = static_cast<size_t>(K / kQK) * kBlockBytes;
    float acc[kTok] = {};
    for (int n = 0; n < N; ++n) {
        const size_t off = n * row_bytes + static_cast<size_t>(k / kQK) * kBlockBytes;
        const float a = block_weight(wg + off, k % kQK), b = block_weight(wu + off, k % kQK);
        for (int t = 0; t < count; ++t) {
            const size_t o = static_cast<size_t>(m0 + t) * N + n;
            acc[t] = fmaf(dg[o], a, fmaf(du[o], b, acc[t]));
        }
    }
    for (int t = 0; t < count; ++t)
        dx[static_cast<size_t>(m0 + t) * K + k] = from_float<__nv_bfloat16>(acc[t]);
}

// t[i, r] = s_a sum_k A_a[r, k] x[i, k], one warp per (token, r); tokens without
// an adapter get zeros.  The first block also counts the ids out of range.
template <typename T>
__global__ void __launch_bounds__(256)
lora_shrink_kernel(const T* __restrict__ x, const __nv_bfloat16* __restrict__ a,
                   const float* __restrict__ scales, const int* __restrict__ ids,
                   float* __restrict__ t, unsigned int* __restrict__ bad_ids, int M, int K, int R,
                   int n_adapters) {
    pdl_allow_dependents();
    const int i = blockIdx.y;
    const int r = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (bad_ids != nullptr && blockIdx.x == 0 && i == 0 && threadIdx.x < 32) {
        unsigned int bad = 0;
        for (int c = lane; c < M; c += 32) bad += ids[c] < -1 || ids[c] >= n_adapters;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) bad += __shfl_xor_sync(0xFFFFFFFFu, bad, o);
        if (lane == 0) *bad_ids = bad;
    }
    if (r >= R) return;
    const int id = ids[i];
    float acc = 0.f;
    if (id >= 0 && id < n_adapters) {
        const __nv_bfloat16* row = a + (static_cast<size_t>(id) * R + r) * K;
        for (int k = lane; k < K; k += 32)
            acc = fmaf(to_float(row[k]), to_float(x[static_cast<size_t>(i) * K + k]), acc);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
        if (scales != nullptr) acc *= scales[id];
    }
    if (lane == 0) t[static_cast<size_t>(i) * R + r] = acc;
}

template <typename T>
__global__ void __launch_bounds__(256)
lora_rows_kernel(const T* __restrict__ x, const uint8_t* __restrict__ w,
                 const __nv_bfloat16* __restrict__ b, const int* __restrict__ ids,
                 const float* __restrict__ t, T* __restrict__ y, int M, int N, int K, int R,
                 int n_adapters) {
    const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (n >= N) return;
    const uint8_t* row = w + static_cast<size_t>(n) * (K / kQK) * kBlockBytes;
    for (int m0 = 0; m0 < M; m0 += kTok) {
        const int count = min(kTok, M - m0);
        float acc[kTok];
        row_dots(x, row, K, m0, count, acc);
        if ((threadIdx.x & 31) == 0)
            for (int c = 0; c < count; ++c) {
                const int m = m0 + c, id = ids[m];
                float v = acc[c];
                if (id >= 0 && id < n_adapters) {
                    const __nv_bfloat16* br = b + (static_cast<size_t>(id) * N + n) * R;
                    for (int r = 0; r < R; ++r)
                        v = fmaf(to_float(br[r]), t[static_cast<size_t>(m) * R + r], v);
                } else if (id != -1) {
                    v = 0.f;  // an id out of range: a zero row, counted by the first kernel
                }
                y[static_cast<size_t>(m) * N + n] = from_float<T>(v);
            }
    }
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

bool ffn_rows_path(int m, bool bf16) { return m <= (bf16 ? 16 : 8); }

size_t gated_workspace_bytes(const GatedArgs&) { return 0; }

cudaError_t launch_gated(const GatedArgs& a, void*, cudaStream_t stream) {
    if (!a.tensor) return launch_gated_rows(a, stream);
    const int blocks = (a.N + 7) / 8;
    if (a.bf16)
        gated_rows_kernel<<<blocks, 256, 0, stream>>>(
            static_cast<const __nv_bfloat16*>(a.x), a.wg, a.wu, static_cast<__nv_bfloat16*>(a.h),
            static_cast<__nv_bfloat16*>(a.gate), static_cast<__nv_bfloat16*>(a.up), a.M, a.N, a.K,
            a.act);
    else
        gated_rows_kernel<<<blocks, 256, 0, stream>>>(
            static_cast<const float*>(a.x), a.wg, a.wu, static_cast<float*>(a.h),
            static_cast<float*>(a.gate), static_cast<float*>(a.up), a.M, a.N, a.K, a.act);
    return cudaGetLastError();
}

size_t gated_backward_workspace_bytes(const GatedBackwardArgs& a) {
    return 2 * align256(static_cast<size_t>(a.M) * a.N * 4);
}

cudaError_t launch_gated_backward(const GatedBackwardArgs& a, void* workspace, cudaStream_t stream) {
    const size_t count = static_cast<size_t>(a.M) * a.N;
    float* dg = static_cast<float*>(workspace);
    float* du = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align256(count * 4));
    const size_t blocks = std::min<size_t>((count + 255) / 256, static_cast<size_t>(a.sm_count) * 8);
    gated_grad_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
        a.dh, a.gate, a.up, dg, du, a.dgate, a.dup, count, a.act);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    gated_dx_kernel<<<dim3(a.K / 128, (a.M + kTok - 1) / kTok), 128, 0, stream>>>(
        dg, du, a.wg, a.wu, a.dx, a.M, a.N, a.K);
    return cudaGetLastError();
}

size_t lora_workspace_bytes(const LoraArgs& a) { return static_cast<size_t>(a.M) * a.R * 4; }

template <typename T>
static cudaError_t launch_lora_as(const LoraArgs& a, void* workspace, cudaStream_t stream) {
    float* t = static_cast<float*>(workspace);
    lora_shrink_kernel<<<dim3((a.R + 7) / 8, a.M), 256, 0, stream>>>(
        static_cast<const T*>(a.x), a.a, a.scales, a.ids, t, a.bad_ids, a.M, a.K, a.R, a.n_adapters);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (!a.tensor) return launch_lora_rows(a, t, stream);
    lora_rows_kernel<<<(a.N + 7) / 8, 256, 0, stream>>>(
        static_cast<const T*>(a.x), a.w, a.b, a.ids, t, static_cast<T*>(a.y), a.M, a.N, a.K, a.R,
        a.n_adapters);
    return cudaGetLastError();
}

cudaError_t launch_lora(const LoraArgs& a, void* workspace, cudaStream_t stream) {
    return a.bf16 ? launch_lora_as<__nv_bfloat16>(a, workspace, stream)
                  : launch_lora_as<float>(a, workspace, stream);
}

}  // namespace q2k
