// The host side of the tensor path of the feed-forward operators: workspaces, the
// kernels that run before the product (f32 tokens' image, gradients of the activations,
// the table of tokens in segments) and the product's launches.
#include <algorithm>
#include <atomic>
#include <mutex>
#include <type_traits>

#include "q2k_ffn_tc.cuh"

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

bool make_weight_map(CUtensorMap* map, const uint8_t* w, int N, int K, int rows, int group,
                     int matrices) {
    const uint64_t row_bytes = static_cast<uint64_t>(K / kQK) * kBlockBytes * group;
    if (matrices > 1 && N % group != 0) return false;  // (the matrices do not start with a group)
    N /= group;
    if (N == 0) return false;
    if (row_bytes % 16 != 0 || (reinterpret_cast<uintptr_t>(w) & 15) != 0) return false;
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    const cuuint64_t dims[3] = {row_bytes, static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(std::max(matrices, 1))};
    const cuuint64_t strides[2] = {row_bytes, row_bytes * static_cast<cuuint64_t>(N)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(kBoxBytes), static_cast<cuuint32_t>(rows), 1};
    const cuuint32_t elem[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, matrices > 0 ? 3 : 2, const_cast<uint8_t*>(w), dims, strides, box,
                  elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc

namespace {

using namespace tc;

// x (f32 [M, K]) -> the bf16 tile image; rows past M up to a multiple of 16 are
// zeros (their sums are dropped, but the MMA reads them).  One thread writes
// 16-byte chunks, four per pass with their loads issued together.
__global__ void __launch_bounds__(256)
x_image_kernel(const float* __restrict__ x, uint8_t* __restrict__ xa, int M, int K, size_t chunks,
               unsigned int* __restrict__ counts, int n_counts) {
    pdl_allow_dependents();
    if (blockIdx.x == 0)
        for (int c = threadIdx.x; c < n_counts; c += blockDim.x) counts[c] = 0u;
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

// The token tiles of segments [offsets[e], offsets[e + 1]): {segment, first token,
// tokens} of `rows` tokens at most, segment after segment.  Offsets that do not ascend
// within 0 .. M give other tiles, but none outside the tokens, and not more than there
// is room for.  f32 tokens are rounded to bf16 on the way, by all CTAs (the first
// makes the table).
constexpr int kTableThreads = 1024;
struct TableArgs {
    const int* offsets;
    int segments, M, rows, capacity;
    int4* table;
    int* count;
    const float* x;
    __nv_bfloat16* xb;
    size_t chunks;  // of eight values
};

__device__ __forceinline__ void make_table(const TableArgs& p, int* first) {  // first: [segments + 1]
    __shared__ int sums[kTableThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x;
    int carry = 0;
    for (int e0 = 0; e0 < p.segments; e0 += threads) {
        const int e = e0 + tid;
        const int tiles = e < p.segments ? tiles_of(segment_tokens(p.offsets, e, p.M), p.rows) : 0;
        int sum = tiles;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, sum, d);
            if (lane >= d) sum += v;
        }
        if (lane == 31) sums[warp] = sum;
        __syncthreads();
        int before = carry, all = carry;
        for (int w = 0; w < threads / 32; ++w) {
            before += w < warp ? sums[w] : 0;
            all += sums[w];
        }
        // (kept at the room there is: no sum of lengths overflows)
        if (e < p.segments) first[e] = min(before + sum - tiles, p.capacity);
        carry = min(all, p.capacity);
        __syncthreads();
    }
    if (tid == 0) {
        first[p.segments] = carry;
        *p.count = carry;
    }
    __syncthreads();
    for (int t = tid; t < carry; t += threads) {
        const TableEntry entry = table_entry(first, p.offsets, p.segments, p.M, p.rows, t);
        p.table[t] = make_int4(entry.segment, entry.first, entry.tokens, 0);
    }
}

__global__ void __launch_bounds__(kTableThreads) table_kernel(TableArgs p) {
    extern __shared__ int table_smem[];
    pdl_allow_dependents();
    pdl_wait_prerequisites();
    if (blockIdx.x == 0) make_table(p, table_smem);
    if (p.xb == nullptr) return;
    for (size_t i = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < p.chunks;
         i += static_cast<size_t>(gridDim.x) * blockDim.x) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p.x) + 2 * i);
        const float4 b = __ldg(reinterpret_cast<const float4*>(p.x) + 2 * i + 1);
        reinterpret_cast<uint4*>(p.xb)[i] = make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w),
                                                       pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
    }
}

// dg = dh u act'(g) and du = dh act(g), rounded to bf16 as the MMA's operands:
// rows of `pitch` (the products' token matrices) and, where the caller's own
// rows are not those, of N.  A thread takes kEach consecutive n of a row: eight where
// rows are whole 16 bytes, else two, since it then loads them one by one (512 tokens of
// 4999x2816, the whole backward pass, us: eight 55.2, two 44.9).  With segments
// a CTA of its own makes the table meanwhile (225 rows of 10 segments, the whole backward
// pass of 1001x1280, us: with a kernel of its own 24.8, so 23.2).
template <bool kSeg, int kEach>
__global__ void __launch_bounds__(256)
grad_kernel(const __nv_bfloat16* __restrict__ dh, const __nv_bfloat16* __restrict__ gate,
            const __nv_bfloat16* __restrict__ up, __nv_bfloat16* __restrict__ dg,
            __nv_bfloat16* __restrict__ du, int pitch, __nv_bfloat16* __restrict__ dgate,
            __nv_bfloat16* __restrict__ dup, int M, int N, int act,
            unsigned int* __restrict__ counts, int n_counts, TableArgs t) {
    extern __shared__ int table_smem[];
    pdl_allow_dependents();
    int first = 0, block = blockIdx.x, blocks = gridDim.x;
    if constexpr (kSeg) {
        if (block == 0) {
            make_table(t, table_smem);
            return;
        }
        --block;
        --blocks;
        // tokens in segments: from the first to the last one's end
        first = held(t.offsets[0], 0, M);
        M = held(t.offsets[t.segments], 0, M);
    }
    if (block == 0)
        for (int c = threadIdx.x; c < n_counts; c += blockDim.x) counts[c] = 0u;
    const int per_row = pitch / kEach;  // (pitch: a multiple of eight)
    const size_t chunks = static_cast<size_t>(M) * per_row;
    for (size_t id = static_cast<size_t>(first) * per_row + static_cast<size_t>(block) * blockDim.x + threadIdx.x;
         id < chunks; id += static_cast<size_t>(blocks) * blockDim.x) {
        const int m = static_cast<int>(id / per_row);
        const int n = kEach * static_cast<int>(id - static_cast<size_t>(m) * per_row);
        const size_t at = static_cast<size_t>(m) * N + n;
        alignas(16) __nv_bfloat16 h[kEach], g[kEach], u[kEach];
        alignas(16) __nv_bfloat16 a[kEach], b[kEach];
        if constexpr (kEach == 8) {
            *reinterpret_cast<uint4*>(h) = __ldg(reinterpret_cast<const uint4*>(dh + at));
            *reinterpret_cast<uint4*>(g) = __ldg(reinterpret_cast<const uint4*>(gate + at));
            *reinterpret_cast<uint4*>(u) = __ldg(reinterpret_cast<const uint4*>(up + at));
        } else {
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const bool ok = n + e < N;
                h[e] = ok ? dh[at + e] : __float2bfloat16_rn(0.f);
                g[e] = ok ? gate[at + e] : __float2bfloat16_rn(0.f);
                u[e] = ok ? up[at + e] : __float2bfloat16_rn(0.f);
            }
        }
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            float value, slope;
            act_value_slope<true>(to_float(g[e]), act, value, slope);
            a[e] = __float2bfloat16_rn(to_float(h[e]) * to_float(u[e]) * slope);
            b[e] = __float2bfloat16_rn(to_float(h[e]) * value);
        }
        const size_t to = static_cast<size_t>(m) * pitch + n;
        using W = std::conditional_t<kEach == 8, uint4, uint32_t>;
        *reinterpret_cast<W*>(dg + to) = *reinterpret_cast<const W*>(a);
        *reinterpret_cast<W*>(du + to) = *reinterpret_cast<const W*>(b);
        if (dgate != nullptr) {
            for (int e = 0; e < kEach && n + e < N; ++e) {
                dgate[at + e] = a[e];
                dup[at + e] = b[e];
            }
        }
    }
}

// dz = dy act'(z) for one matrix, and its sums over the tokens (of each segment):
// dbias.  A CTA takes 128 columns (a lane four of them) and a share of a segment's
// tokens, a warp every eighth, four at once (lanes of eight columns, two tokens at once,
// the whole backward pass, us: 225 rows of 10 segments of 1001x1280 25.2, so 17.4; 4096 of
// 64 of 2048x2048 112.4, so 109; 2048 tokens of 14336x4096 198, so 194; 512 the same); a cluster's CTAs share a segment and add their sums in
// order.  dz goes to rows of `pitch`, and to the caller's own rows where those differ;
// without an activation dz is dy, and only sums, or rows of `pitch`, may be asked for.
// A sum takes dz before it is rounded.  With segments the first CTA of a row of CTAs in
// front makes the table meanwhile.
struct LinearGradArgs {
    const __nv_bfloat16* dy;
    const __nv_bfloat16* z;   // with an activation
    __nv_bfloat16* to;        // rows of `pitch`, or null
    __nv_bfloat16* dz;        // the caller's, or null
    float* dbias;             // [segments][N], or null
    TableArgs table;          // of the segments (offsets null: one of M tokens)
    unsigned int* counts;
    int n_counts;
    int M, N, pitch;
    int shares;               // CTAs of a segment and kGradCols columns (with dbias: a cluster)
};
constexpr int kGradCols = 128, kGradWarps = 8, kGradAtOnce = 4;
static_assert(kGradCols == 32 * kGradEach, "a warp's columns");

// act'(g) in few instructions, which bound this kernel beside its loads (7.3 million
// values of gelu: 15.7 us with act_value_slope, 12.2 so): with p the logistic of z as
// there, p + g (1 - p) p z' = p (1 + q - p q), q = g z'; e^-z as a power of two.  Past
// the bounds p is 0 or 1 in f32, and q only has to stay finite (a NaN passes).
template <int kAct>
__device__ __forceinline__ float act_slope(float g) {
    constexpr float kC = 1.5957691216057308f, kA = 0.044715f, kLog2e = 1.4426950408889634f;
    constexpr bool gelu = kAct == kActGelu;
    constexpr float top = gelu ? 30.f : 128.f;
    float c, e, r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(g), "f"(-top));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(c), "f"(top));
    float q = c, z = -kLog2e;
    if (gelu) {
        const float s = c * c;
        z = fmaf(-kLog2e * kC * kA, s, -kLog2e * kC);
        q = c * fmaf(3.f * kA * kC, s, kC);
    }
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(c * z));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return fmaf(r, fmaf(-r, q, q), r);
}

// A lane's bf16 values of a row.
struct Lane {
    union {
        uint2 word;
        uint32_t bits[kGradEach / 2];
        __nv_bfloat16 value[kGradEach];
    };
    __device__ __forceinline__ Lane() : word() {}
    __device__ __forceinline__ float get(int e) const {
        return __uint_as_float(e & 1 ? bits[e / 2] & 0xFFFF0000u : bits[e / 2] << 16);
    }
};

template <int kAct>
__global__ void __launch_bounds__(32 * kGradWarps, 4) linear_grad_kernel(LinearGradArgs p) {
    extern __shared__ int table_smem[];
    __shared__ float red[kGradWarps][kGradCols];
    __shared__ float part[kGradCols];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int share = blockIdx.x % p.shares, n0 = kGradCols * (blockIdx.x / p.shares);
    const bool segments = p.table.offsets != nullptr;
    const int n = n0 + kGradEach * lane, segment = static_cast<int>(blockIdx.y) - segments;
    pdl_wait_prerequisites();
    pdl_allow_dependents();  // (later grids start when all before this one is complete)
    if (segment < 0) {  // (whole clusters)
        if (blockIdx.x == 0) make_table(p.table, table_smem);
        return;
    }
    if (blockIdx.x == 0 && segment == 0)
        for (int c = threadIdx.x; c < p.n_counts; c += blockDim.x) p.counts[c] = 0u;
    const Tokens tokens = segments ? segment_tokens(p.table.offsets, segment, p.M) : Tokens{0, p.M};
    const long long len = tokens.hi - tokens.lo;
    const int lo = tokens.lo + static_cast<int>(len * share / p.shares);
    const int hi = tokens.lo + static_cast<int>(len * (share + 1) / p.shares);
    constexpr bool kZ = kAct != kActNone;
    const bool vec = p.N % kGradEach == 0;
    const int inside = grad_inside(n, p.N);  // (the lane's other columns are zeros)
    float sum[kGradEach] = {};
    for (int m0 = lo + warp; m0 < hi && n < p.pitch; m0 += kGradAtOnce * kGradWarps) {
        Lane g[kGradAtOnce], z[kGradAtOnce];
#pragma unroll
        for (int u = 0; u < kGradAtOnce; ++u) {
            // (a token past the end is the last one again, which counts for nothing)
            const int m = min(m0 + u * kGradWarps, hi - 1);
            const size_t at = static_cast<size_t>(m) * p.N + n;
            if (vec) {
                if (inside == 0) continue;
                g[u].word = __ldg(reinterpret_cast<const uint2*>(p.dy + at));
                if (kZ) z[u].word = __ldg(reinterpret_cast<const uint2*>(p.z + at));
            } else {
#pragma unroll
                for (int e = 0; e < kGradEach; ++e) {
                    const bool ok = e < inside;
                    g[u].value[e] = ok ? p.dy[at + e] : __float2bfloat16_rn(0.f);
                    z[u].value[e] = ok && kZ ? p.z[at + e] : __float2bfloat16_rn(0.f);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kGradAtOnce; ++u) {
            const int m = m0 + u * kGradWarps;
            if (m >= hi) break;
            Lane d;
#pragma unroll
            for (int e = 0; e < kGradEach; e += 2) {
                float v = g[u].get(e), w = g[u].get(e + 1);
                if (kZ) {
                    v *= act_slope<kAct>(z[u].get(e));
                    w *= act_slope<kAct>(z[u].get(e + 1));
                }
                sum[e] += v;
                sum[e + 1] += w;
                d.bits[e / 2] = pack_bf16(v, w);
            }
            if (p.to != nullptr) *reinterpret_cast<uint2*>(p.to + static_cast<size_t>(m) * p.pitch + n) = d.word;
            if (p.dz != nullptr)
                for (int e = 0; e < kGradEach && e < inside; ++e) p.dz[static_cast<size_t>(m) * p.N + n + e] = d.value[e];
        }
    }
    if (p.dbias == nullptr) return;  // (all CTAs alike)
#pragma unroll
    for (int e = 0; e < kGradEach; ++e) red[warp][kGradEach * lane + e] = sum[e];
    __syncthreads();
    float v = 0.f;
    if (threadIdx.x < kGradCols) {
#pragma unroll
        for (int w = 0; w < kGradWarps; ++w) v += red[w][threadIdx.x];
        part[threadIdx.x] = v;
    }
    if (p.shares > 1) {
        __syncwarp();
        cluster_sync();
        if (share == 0 && threadIdx.x < kGradCols) {
            v = 0.f;
            for (int c = 0; c < p.shares; ++c) {
                float w;
                asm volatile(
                    "{\n\t.reg .u32 ra;\n\tmapa.shared::cluster.u32 ra, %1, %2;\n\t"
                    "ld.shared::cluster.f32 %0, [ra];\n\t}"
                    : "=f"(w)
                    : "r"(smem_u32(part + threadIdx.x)), "r"(c)
                    : "memory");
                v += w;
            }
        }
        __syncwarp();
        cluster_sync();  // the sums are read before their CTA leaves
    }
    const int col = n0 + static_cast<int>(threadIdx.x);
    if (share == 0 && threadIdx.x < kGradCols && col < p.N) p.dbias[static_cast<size_t>(segment) * p.N + col] = v;
}

// ---- plan ----------------------------------------------------------------------

size_t plan_bytes(const Plan& p) { return p.partial + p.counts; }
int count_words(const Plan& p) { return static_cast<int>(p.counts / 4); }

size_t image_bytes(int M, int K) {
    return static_cast<size_t>((M + kSuperRows - 1) / kSuperRows) * kSuperRows * K * 2;
}

// The segments of a call's tokens: as many as matrices, or none (offsets null).
struct Segments {
    const int* offsets;
    int count;
};

Plan forward_plan(int M, int N, int K, bool gated, int experts = 0) {
    const int tile_rows = gated ? kRows / 2 : kRows;
    return experts > 0 ? make_segment_plan(M, N, tile_rows, K / kQK, experts)
                       : make_plan(M, N, tile_rows, K / kQK);
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
// The count and the table of tiles.
size_t table_bytes(const Plan& plan) {
    return align256(16 + static_cast<size_t>(plan.tiles / plan.row_units) * sizeof(int4));
}

template <typename Args>
cudaError_t launch_pdl(void (*kernel)(Args), dim3 grid, int threads, size_t smem, int cluster,
                       cudaStream_t stream, const Args& args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args);
}

// The table at `workspace`, of tiles of `rows` tokens.
TableArgs table_args(const Segments& seg, int M, int rows, int capacity, uint8_t* workspace) {
    TableArgs p = {};
    p.offsets = seg.offsets;
    p.segments = seg.count;
    p.M = M;
    p.rows = rows;
    p.capacity = capacity;
    p.count = reinterpret_cast<int*>(workspace);
    p.table = reinterpret_cast<int4*>(workspace + 16);
    return p;
}
TableArgs table_args(const Segments& seg, int M, const Plan& plan, uint8_t* workspace) {
    return table_args(seg, M, plan.x_rows, plan.tiles / plan.row_units, workspace);
}
size_t table_smem_bytes(const Segments& seg) { return (seg.count + 1) * sizeof(int); }

// The table in a kernel of its own; x: f32 tokens that xb gets.
cudaError_t launch_table(TableArgs p, const Segments& seg, const float* x, __nv_bfloat16* xb, int K, int sm_count,
                         cudaStream_t stream) {
    p.x = x;
    p.xb = xb;
    p.chunks = xb != nullptr ? static_cast<size_t>(p.M) * (K / 8) : 0;
    const size_t wanted = (p.chunks + 2 * kTableThreads - 1) / (2 * kTableThreads);
    const unsigned ctas = static_cast<unsigned>(std::min<size_t>(std::max<size_t>(wanted, 1), 2 * sm_count));
    // (few warps meet sooner)
    const int threads = xb != nullptr ? kTableThreads : std::min(kTableThreads, (std::max(seg.count, p.capacity) + 31) & ~31);
    return launch_pdl(table_kernel, dim3(ctas), threads, table_smem_bytes(seg), 1, stream, p);
}

// Workspace of x W^T: plan_bytes, then (f32) the tokens' image; in segments the table,
// then (f32) a bf16 copy of the tokens, since segments begin anywhere.
size_t forward_workspace_bytes(int M, int N, int K, bool gated, bool bf16, int experts) {
    const Plan plan = forward_plan(M, N, K, gated, experts);
    if (experts > 0) return table_bytes(plan) + (bf16 ? 0 : static_cast<size_t>(M) * K * 2);
    return plan_bytes(plan) + (bf16 ? 0 : image_bytes(M, K));
}

// x W^T of tokens in segments.
template <Tc kMode>
cudaError_t launch_segments(TcArgs a, bool bf16, const void* x, void* workspace, int device, int sm_count,
                            cudaStream_t stream, Segments seg) {
    const Plan plan = forward_plan(a.M, a.N, a.K, kMode == Tc::kGated, seg.count);
    a.quads = a.K / kQK;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    __nv_bfloat16* xb = bf16 ? nullptr : reinterpret_cast<__nv_bfloat16*>(ws + table_bytes(plan));
    const cudaError_t e = launch_table(table_args(seg, a.M, plan, ws), seg, static_cast<const float*>(x), xb, a.K,
                                       sm_count, stream);
    if (e != cudaSuccess) return e;
    a.table_count = reinterpret_cast<const int*>(ws);
    a.table = reinterpret_cast<const int4*>(ws + 16);
    a.const_weights = a.tokens_ready = true;  // (the kernel waits before it reads the table)
    return bf16 ? launch_tc<kMode, __nv_bfloat16, true>(a, plan, ws, x, nullptr, a.K, a.K, device, stream,
                                                        seg.count)
                : launch_tc<kMode, float, true>(a, plan, ws, xb, nullptr, a.K, a.K, device, stream, seg.count);
}

// x W^T: bf16 tokens go to the kernel by their own tensor map, f32 tokens by an
// image.  behind_grid: one of this call's own grids (which does not write x, and
// zeroes the counts) is before, and lets its dependents start only when x is
// complete.
template <Tc kMode>
cudaError_t launch_forward(TcArgs a, bool bf16, const void* x, void* workspace, int device,
                           int sm_count, bool behind_grid, cudaStream_t stream) {
    const Plan plan = forward_plan(a.M, a.N, a.K, kMode == Tc::kGated);
    a.quads = a.K / kQK;
    a.tokens_ready = bf16 && behind_grid;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    unsigned int* counts = reinterpret_cast<unsigned int*>(ws + plan.partial);
    if (bf16) {
        if (!behind_grid && plan.counts != 0) {
            const cudaError_t e = cudaMemsetAsync(counts, 0, plan.counts, stream);
            if (e != cudaSuccess) return e;
        }
        return launch_tc<kMode, __nv_bfloat16, false>(a, plan, ws, x, nullptr, a.K, a.K, device, stream, 1);
    }
    uint8_t* image = ws + plan_bytes(plan);
    a.xa = image;
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, x_image_kernel, static_cast<const float*>(x), image,
                                             a.M, a.K, chunks, counts, count_words(plan));
    if (e != cudaSuccess) return e;
    return launch_tc<kMode, float, false>(a, plan, ws, nullptr, nullptr, 0, 0, device, stream, 1);
}

// Columns of one of the token matrices as the product's K: over both of two, or in the
// one, whole fours of stages.
int backward_cols(int N, int matrices) {
    const int unit = 4 / matrices * kStageK;
    return (N + unit - 1) / unit * unit;
}
// Their rows' pitch: the caller's own when those are whole 16 bytes.
int backward_pitch(int N) { return (N + 7) & ~7; }

}  // namespace

size_t ffn_table_bytes(int M, int segments, int rows) {
    return align256(16 + static_cast<size_t>(segment_tiles(M, segments, rows)) * sizeof(int4));
}

cudaError_t launch_ffn_table(const int* offsets, int segments, int M, int rows, void* workspace,
                             int sm_count, cudaStream_t stream) {
    const Segments seg = {offsets, segments};
    return launch_table(table_args(seg, M, rows, segment_tiles(M, segments, rows), static_cast<uint8_t*>(workspace)),
                        seg, nullptr, nullptr, 0, sm_count, stream);
}

size_t gated_tc_workspace_bytes(const GatedArgs& a) {
    return forward_workspace_bytes(a.M, a.N, a.K, true, a.bf16, a.n_experts);
}

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
    if (a.n_experts > 0)
        return launch_segments<Tc::kGated>(t, a.bf16, a.x, workspace, a.device, a.sm_count, stream,
                                           {a.offsets, a.n_experts});
    return launch_forward<Tc::kGated>(t, a.bf16, a.x, workspace, a.device, a.sm_count, false, stream);
}

size_t linear_tc_workspace_bytes(const LinearArgs& a) {
    return forward_workspace_bytes(a.M, a.N, a.K, false, a.bf16, a.n_experts);
}

cudaError_t launch_linear_tc(const LinearArgs& a, void* workspace, cudaStream_t stream) {
    TcArgs t = {};
    t.w0 = t.w1 = a.w;
    t.M = a.M;
    t.N = a.N;
    t.K = a.K;
    t.const_weights = a.const_weights;
    t.bias = a.bias;
    t.residual = a.residual;
    t.y = a.y;
    t.z = a.z;
    t.act = a.act;
    if (a.n_experts > 0)
        return launch_segments<Tc::kLinear>(t, a.bf16, a.x, workspace, a.device, a.sm_count, stream,
                                            {a.offsets, a.n_experts});
    return launch_forward<Tc::kLinear>(t, a.bf16, a.x, workspace, a.device, a.sm_count, false, stream);
}

size_t lora_tc_workspace_bytes(const LoraArgs& a) {
    return forward_workspace_bytes(a.M, a.N, a.K, false, a.bf16, 0);
}

void lora_tc_counts(const LoraArgs& a, void* workspace, unsigned int** counts, int* n_counts) {
    const Plan plan = forward_plan(a.M, a.N, a.K, false);
    *counts = reinterpret_cast<unsigned int*>(static_cast<uint8_t*>(workspace) + plan.partial);
    *n_counts = count_words(plan);
}

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

// Workspace: plan_bytes; then dg and du, unless the caller takes them in rows of
// whole 16 bytes.
static bool backward_in_place(const GatedBackwardArgs& a) {
    return a.dgate != nullptr && backward_pitch(a.N) == a.N;
}
static size_t backward_matrix_bytes(int M, int N) {
    return align256(static_cast<size_t>(M) * backward_pitch(N) * 2);
}
static Plan backward_plan(int M, int N, int K, int matrices, int experts) {
    const int quads = matrices * backward_cols(N, matrices) / (4 * kStageK);
    return experts > 0 ? make_segment_plan(M, K, kRows, quads, experts) : make_plan(M, K, kRows, quads);
}
// Of the product alone: plan_bytes, or the table.
static size_t backward_plan_bytes(const Plan& plan, int experts) {
    return experts > 0 ? table_bytes(plan) : plan_bytes(plan);
}
size_t gated_backward_workspace_bytes(const GatedBackwardArgs& a) {
    return backward_plan_bytes(backward_plan(a.M, a.N, a.K, 2, a.n_experts), a.n_experts) +
           (backward_in_place(a) ? 0 : 2 * backward_matrix_bytes(a.M, a.N));
}

// dx = sum over the matrices (w1: the second, or w0 again) of their tokens d0 (and d1),
// rows of `pitch`.  The counts are zeroed.  const_weights: the grid before started when
// all before it was complete.
static cudaError_t launch_backward_product(const uint8_t* w0, const uint8_t* w1, const void* d0,
                                           const void* d1, __nv_bfloat16* dx, const Plan& plan, int M, int N,
                                           int K, int matrices, int pitch, Segments seg, bool const_weights,
                                           uint8_t* ws, int device, cudaStream_t stream) {
    TcArgs t = {};
    t.w0 = w0;
    t.w1 = w1;
    t.M = M;
    t.N = N;
    t.K = K;
    t.const_weights = const_weights;
    t.half_stages = backward_cols(N, matrices) / kStageK;
    t.quads = matrices * t.half_stages / 4;
    t.y = dx;
    if (seg.count > 0) {
        t.table_count = reinterpret_cast<const int*>(ws);
        t.table = reinterpret_cast<const int4*>(ws + 16);
    }
    return seg.count > 0 ? launch_tc<Tc::kBackward, __nv_bfloat16, true>(t, plan, ws, d0, d1, N, pitch, device,
                                                                         stream, seg.count)
                         : launch_tc<Tc::kBackward, __nv_bfloat16, false>(t, plan, ws, d0, d1, N, pitch, device,
                                                                          stream, 1);
}

cudaError_t launch_gated_backward(const GatedBackwardArgs& a, void* workspace, cudaStream_t stream) {
    const Segments seg = {a.offsets, a.n_experts};
    const Plan plan = backward_plan(a.M, a.N, a.K, 2, seg.count);
    const int pitch = backward_pitch(a.N);
    const bool own = backward_in_place(a);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    uint8_t* copies = ws + backward_plan_bytes(plan, seg.count);
    __nv_bfloat16* dg = own ? a.dgate : reinterpret_cast<__nv_bfloat16*>(copies);
    __nv_bfloat16* du = own ? a.dup
                            : reinterpret_cast<__nv_bfloat16*>(copies + backward_matrix_bytes(a.M, a.N));
    const bool whole = (a.N & 7) == 0, in_segments = seg.count > 0;
    const size_t chunks = static_cast<size_t>(a.M) * (pitch / (whole ? 8 : 2));
    const unsigned blocks =
        static_cast<unsigned>(std::min<size_t>((chunks + 255) / 256, static_cast<size_t>(a.sm_count) * 8));
    const TableArgs table = in_segments ? table_args(seg, a.M, plan, ws) : TableArgs{};
    const auto kernel = in_segments ? (whole ? grad_kernel<true, 8> : grad_kernel<true, 2>)
                                    : (whole ? grad_kernel<false, 8> : grad_kernel<false, 2>);
    kernel<<<blocks + in_segments, 256, in_segments ? table_smem_bytes(seg) : 0, stream>>>(
        a.dh, a.gate, a.up, dg, du, pitch, own ? nullptr : a.dgate, own ? nullptr : a.dup, a.M, a.N,
        a.act, reinterpret_cast<unsigned int*>(ws + plan.partial), count_words(plan), table);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_backward_product(a.wg, a.wu, dg, du, a.dx, plan, a.M, a.N, a.K, 2, pitch, seg, true, ws,
                                   a.device, stream);
}

// Workspace: the product's, then dz where it is neither the caller's own (dz given, or
// dy without an activation) nor in rows of whole 16 bytes.
static bool linear_backward_in_place(const LinearBackwardArgs& a) {
    return backward_pitch(a.N) == a.N && (a.act == kActNone || a.dz != nullptr);
}
size_t linear_backward_workspace_bytes(const LinearBackwardArgs& a) {
    return backward_plan_bytes(backward_plan(a.M, a.N, a.K, 1, a.n_experts), a.n_experts) +
           (linear_backward_in_place(a) ? 0 : backward_matrix_bytes(a.M, a.N));
}

cudaError_t launch_linear_backward(const LinearBackwardArgs& a, void* workspace, cudaStream_t stream) {
    const Segments seg = {a.offsets, a.n_experts};
    const Plan plan = backward_plan(a.M, a.N, a.K, 1, seg.count);
    const bool own = linear_backward_in_place(a);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaError_t e = cudaSuccess;
    LinearGradArgs g = {};
    g.dy = a.dy;
    g.z = a.act == kActNone ? nullptr : a.z;
    g.M = a.M;
    g.N = a.N;
    g.pitch = backward_pitch(a.N);
    if (seg.count > 0) g.table = table_args(seg, a.M, plan, ws);
    g.dbias = a.dbias;
    g.counts = reinterpret_cast<unsigned int*>(ws + plan.partial);
    g.n_counts = count_words(plan);
    const __nv_bfloat16* d0 = a.dy;
    if (!own) {
        d0 = g.to = reinterpret_cast<__nv_bfloat16*>(ws + backward_plan_bytes(plan, seg.count));
        g.dz = a.dz;
    } else if (g.z != nullptr) {
        d0 = g.to = a.dz;
    }
    const bool grads = g.to != nullptr || g.dbias != nullptr;
    if (grads) {
        // a warp's rows at once are the least a share is worth; a cluster's eight at most
        // where sums meet
        const int segments = std::max(1, seg.count);
        const int rows = std::max(1, a.M / segments);
        const int strips = (g.pitch + kGradCols - 1) / kGradCols;
        const int most = g.dbias != nullptr ? kMaxParts : std::max(1, 16 * a.sm_count / strips);
        g.shares = std::min(most, std::max(1, rows / (kGradAtOnce * kGradWarps)));
        e = launch_pdl(a.act == kActNone   ? linear_grad_kernel<kActNone>
                       : a.act == kActGelu ? linear_grad_kernel<kActGelu>
                                           : linear_grad_kernel<kActSilu>,
                       dim3(strips * g.shares, segments + (seg.count > 0)), 32 * kGradWarps,
                       seg.count > 0 ? table_smem_bytes(seg) : 0, g.dbias != nullptr ? g.shares : 1, stream, g);
    } else if (seg.count > 0) {
        e = launch_table(table_args(seg, a.M, plan, ws), seg, nullptr, nullptr, 0, a.sm_count, stream);
    } else if (plan.counts != 0) {
        e = cudaMemsetAsync(ws + plan.partial, 0, plan.counts, stream);
    }
    if (e != cudaSuccess) return e;
    return launch_backward_product(a.w, a.w, d0, d0, a.dx, plan, a.M, a.N, a.K, 1, g.pitch, seg,
                                   grads || seg.count > 0, ws, a.device, stream);
}

// (the address of a module's variable: the same for a device as long as it lasts)
cudaError_t ffn_error_word(int device, unsigned int** word) {
    static std::atomic<unsigned int*> known[64] = {};
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    *word = known[device].load(std::memory_order_acquire);
    if (*word != nullptr) return cudaSuccess;
    void* at = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&at, g_ffn_error);
    if (e != cudaSuccess) return e;
    *word = static_cast<unsigned int*>(at);
    known[device].store(*word, std::memory_order_release);
    return cudaSuccess;
}

// The error words: this file's, and those of the tensor kernel's files (added while the
// library is loaded, only read after).
constexpr int kMaxErrorWords = 16;
static const void* g_tc_error_words[kMaxErrorWords];
static int g_tc_error_count;

bool add_tc_error_word(const void* symbol) {
    if (g_tc_error_count == kMaxErrorWords) return false;
    g_tc_error_words[g_tc_error_count++] = symbol;
    return true;
}

cudaError_t read_and_clear_ffn_error(uint32_t* out, cudaStream_t stream) {
    unsigned int bits[kMaxErrorWords + 1] = {};
    const unsigned int zero = 0;
    auto word = [](int i) { return i < g_tc_error_count ? g_tc_error_words[i] : &g_ffn_error; };
    for (int i = 0; i <= g_tc_error_count; ++i) {
        const cudaError_t e = cudaMemcpyFromSymbolAsync(bits + i, word(i), sizeof(unsigned int), 0,
                                                        cudaMemcpyDeviceToHost, stream);
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return e;
    *out = 0;
    for (int i = 0; i <= g_tc_error_count; ++i) {
        *out |= bits[i];
        if (bits[i] == 0) continue;
        e = cudaMemcpyToSymbolAsync(word(i), &zero, sizeof(unsigned int), 0, cudaMemcpyHostToDevice, stream);
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace q2k
