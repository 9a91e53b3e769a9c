// Tokens to their experts and back: the places of a router's choices in expert
// order, rows of activations moved there, and the experts' rows brought back to
// their tokens with the router's weights; and the gradients of both moves.
//
//   route    rows[i] = #{j: e_j < e_i, or e_j = e_i and j < i}   (a stable counting sort)
//   sort     xs[rows[t, s]] = x[t];                dx[t] = sum_s dxs[rows[t, s]]
//   combine  y[t] = r[t] + sum_s w[t, s] ys[rows[t, s]];
//            dys[rows[t, s]] = w[t, s] dy[t],  dw[t, s] = <dy[t], ys[rows[t, s]]>
//
// The moves do next to no arithmetic: HBM bounds them, and the latency of a
// dependent load or two where there are few tokens.  All of them go by tokens: the
// token's row is read once and its top_k places follow from `rows`, so that every
// result has one writer and sums have a fixed order, without atomics.  Sums are f32
// (a token's over its slots in the order of the slots), rounded once.
//
// `rows` is a permutation of all n_tokens * top_k places: choices without an expert
// come last, from offsets[n_experts] on.  Their places are written as zeros and
// never read.
//
// Each kernel lets the next grid start once all before itself are complete: a call
// behind it that reads its weights early then finds them written.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "q2k_device.cuh"
#include "q2k_ffn.cuh"
#include "q2k_internal.h"

namespace q2k {

namespace {

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t load_cluster_u32(uint32_t addr, uint32_t rank) {
    uint32_t v;
    asm volatile(
        "{\n\t.reg .u32 ra;\n\tmapa.shared::cluster.u32 ra, %1, %2;\n\t"
        "ld.shared::cluster.u32 %0, [ra];\n\t}"
        : "=r"(v)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

// ---- route -----------------------------------------------------------------------
//
// One cluster: each CTA takes a run of the choices, each warp a run of the CTA's, 32
// at a time, with counts of its own per expert (bins).  A first walk counts; the
// counts become places (over the warps, the CTAs of the cluster, the experts); a
// second walk gives each choice its place, its rank among the 32 from the mask of
// those with the same expert, which a ballot for each bit of the expert gives (262144
// choices of 64 experts, us: with `match` in both walks 62, counting by atomics in
// shared memory 40, with ballots 33).  Nothing depends on the order in which warps
// run.
constexpr int kRouteMaxCtas = 8;
constexpr int kRouteWarps = 16, kRouteWarpsMany = 8;  // (more bins than kRouteFewBins)
constexpr int kRouteFewBins = 2048;
constexpr int kRouteEach = 32;

struct RouteArgs {
    const int* ids;
    int* rows;
    int* order;
    int* offsets;
    unsigned int* bad_ids;
    int routes, experts;
    int bits;  // of an expert's number, and of `experts`
    int each;  // choices of a warp, a multiple of 32
};

__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(RouteArgs p) {
    extern __shared__ int route_smem[];
    const int bins = p.experts + 1;  // the last: no expert
    const int tid = threadIdx.x, threads = blockDim.x, warps = threads >> 5;
    const int warp = tid >> 5, lane = tid & 31;
    const int ctas = gridDim.x, rank = blockIdx.x;
    int* count = route_smem;               // [warps][bins]
    int* total = count + warps * bins;     // [bins + 1]: this CTA's, and its bad ids
    int* start = total + bins + 1;         // [bins]
    for (int i = tid; i < (warps + 1) * bins + 1; i += threads) count[i] = 0;
    pdl_wait_prerequisites();
    pdl_allow_dependents();
    __syncthreads();
    const int first = (rank * warps + warp) * p.each;
    const int last = min(p.routes, first + p.each);
    int* mine = count + warp * bins;
    int bad = 0;
    constexpr int kAhead = 4;
    int id[kAhead];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = base + 32 * u + lane;
            id[u] = i < last ? __ldg(p.ids + i) : -2;
        }
    };
    for (int base = first; base < last; base += 32 * kAhead) {
        load(base);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const bool in = base + 32 * u + lane < last;
            const bool known = static_cast<unsigned>(id[u]) < static_cast<unsigned>(p.experts);
            bad += in && !known && id[u] != -1;
            if (in) atomicAdd(mine + (known ? id[u] : p.experts), 1);  // (a count: any order)
        }
    }
    bad = __reduce_add_sync(0xFFFFFFFFu, bad);
    if (lane == 0 && bad != 0) atomicAdd(total + bins, bad);  // (a count: any order)
    __syncthreads();
    // over the warps
    for (int e = tid; e < bins; e += threads) {
        int sum = 0;
        for (int w = 0; w < warps; ++w) {
            const int c = count[w * bins + e];
            count[w * bins + e] = sum;
            sum += c;
        }
        total[e] = sum;
    }
    // over the cluster's CTAs: those before this one into its counts, all into start
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    for (int e = tid; e < bins; e += threads) {
        int before = 0, all = 0;
        if (ctas > 1) {
            for (int c = 0; c < ctas; ++c) {
                const int v = static_cast<int>(load_cluster_u32(smem_u32(total + e), c));
                before += c < rank ? v : 0;
                all += v;
            }
        } else {
            all = total[e];
        }
        start[e] = all;
        for (int w = 0; w < warps; ++w) count[w * bins + e] += before;
    }
    if (rank == 0 && tid == 0 && p.bad_ids != nullptr) {
        unsigned n = 0;
        for (int c = 0; c < ctas; ++c)
            n += ctas > 1 ? load_cluster_u32(smem_u32(total + bins), c) : static_cast<unsigned>(total[bins]);
        *p.bad_ids = n;
    }
    __syncthreads();
    // over the experts
    if (warp == 0) {
        int carry = 0;
        for (int e0 = 0; e0 < bins; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < bins ? start[e] : 0;
            int sum = c;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, sum, d);
                if (lane >= d) sum += v;
            }
            if (e < bins) start[e] = carry + sum - c;
            if (e < bins && rank == 0) p.offsets[e] = carry + sum - c;
            carry += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
    }
    if (ctas > 1) cluster_arrive();  // (the others' totals are read)
    __syncthreads();
    for (int base = first; base < last; base += 32 * kAhead) {
        if (p.each > 32 * kAhead) load(base);  // (else they are here)
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = base + 32 * u + lane;
            const bool known = static_cast<unsigned>(id[u]) < static_cast<unsigned>(p.experts);
            const int key = i >= last ? -1 : known ? id[u] : p.experts;
            unsigned same = __ballot_sync(0xFFFFFFFFu, key >= 0);
            for (int b = 0; b < p.bits; ++b) {
                const unsigned set = __ballot_sync(0xFFFFFFFFu, (key >> b) & 1);
                same &= (key >> b) & 1 ? set : ~set;
            }
            int at = 0;
            if (key >= 0) {
                at = start[key] + mine[key] + __popc(same & ((1u << lane) - 1u));
                p.rows[i] = at;
                p.order[at] = i;
            }
            __syncwarp();
            if (key >= 0 && lane == __ffs(same) - 1) mine[key] += __popc(same);
            __syncwarp();
        }
    }
    if (ctas > 1) cluster_wait();  // no CTA leaves while another may read its totals
}

// ---- moves -----------------------------------------------------------------------

// V neighbouring values of a row, moved as one word of V * sizeof(T) bytes.
template <int kBytes>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<2> { using type = uint16_t; };

template <typename T, int V>
struct Pack {
    using W = typename Word<V * sizeof(T)>::type;
    union {
        W word;
        uint32_t bits[(V * sizeof(T) + 3) / 4];
        uint16_t half[V * sizeof(T) / 2];
    };
    __device__ __forceinline__ Pack() : word() {}
    __device__ __forceinline__ void load(const T* p) { word = __ldg(reinterpret_cast<const W*>(p)); }
    // Load if `in`, without a branch, and where it stands: loads of several rows are then
    // all asked for before the first is used.  (Left to itself the compiler moved each
    // to its use.)
    __device__ __forceinline__ void load_if(const T* p, bool in) {
        const int ok = in;
        if constexpr (sizeof(W) == 16)
            asm volatile(
                "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %5, 0;\n\t"
                "@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                : "+r"(bits[0]), "+r"(bits[1]), "+r"(bits[2]), "+r"(bits[3])
                : "l"(p), "r"(ok));
        else if constexpr (sizeof(W) == 8)
            asm volatile(
                "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %3, 0;\n\t"
                "@p ld.global.nc.v2.u32 {%0, %1}, [%2];\n\t}"
                : "+r"(bits[0]), "+r"(bits[1])
                : "l"(p), "r"(ok));
        else if constexpr (sizeof(W) == 4)
            asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %2, 0;\n\t@p ld.global.nc.u32 %0, [%1];\n\t}"
                         : "+r"(bits[0])
                         : "l"(p), "r"(ok));
        else
            asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %2, 0;\n\t@p ld.global.nc.u16 %0, [%1];\n\t}"
                         : "+h"(half[0])
                         : "l"(p), "r"(ok));
    }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<W*>(p) = word; }
    __device__ __forceinline__ float get(int v) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(bits[v]);
        else return __uint_as_float(static_cast<uint32_t>(half[v]) << 16);
    }
    __device__ __forceinline__ void set(int v, float f) {
        if constexpr (sizeof(T) == 4) bits[v] = __float_as_uint(f);
        else half[v] = __bfloat16_as_ushort(__float2bfloat16_rn(f));
    }
};

struct MoveArgs {
    const void* in;        // x, dxs or ys
    const void* residual;  // or null
    const float* weights;  // [n_tokens * top_k], or null (all 1)
    const int* rows;
    const int* offsets;
    void* out;
    int top_k, routes, experts;
    int width, units;      // of a row: values, words
    int chunks;            // CTAs that share a row
};

constexpr int kMoveThreads = 256;
constexpr int kSlots = 8;  // places taken together: that many loads on their way

// xs[rows[t, s]] = x[t]; a place without an expert gets zeros.  A thread has kW words of
// the row on their way: sixteen bytes (4096 tokens of two rows of 4097 bf16, words of two
// bytes: one 71.6 us, eight 22).
template <typename T, int V, int kW>
__global__ void __launch_bounds__(kMoveThreads) sort_kernel(MoveArgs p) {
    pdl_wait_prerequisites();
    pdl_allow_dependents();
    const int t = blockIdx.x / p.chunks;
    const int u = (blockIdx.x - t * p.chunks) * kW * blockDim.x + threadIdx.x;
    if (u >= p.units) return;
    const T* x = static_cast<const T*>(p.in) + static_cast<size_t>(t) * p.width + static_cast<size_t>(u) * V;
    T* xs = static_cast<T*>(p.out) + static_cast<size_t>(u) * V;
    const int* rows = p.rows + static_cast<size_t>(t) * p.top_k;
    const int step = blockDim.x * V;  // from one of the thread's words to the next
    Pack<T, V> v[kW], none;
    bool in[kW];
#pragma unroll
    for (int w = 0; w < kW; ++w) {
        in[w] = u + w * static_cast<int>(blockDim.x) < p.units;
        v[w].load_if(x + w * step, in[w]);
    }
    const int end = __ldg(p.offsets + p.experts);
    for (int s0 = 0; s0 < p.top_k; s0 += kSlots) {
        int at[kSlots];
#pragma unroll
        for (int s = 0; s < kSlots; ++s) at[s] = s0 + s < p.top_k ? __ldg(rows + s0 + s) : -1;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            if (static_cast<unsigned>(at[s]) >= static_cast<unsigned>(p.routes)) continue;
            T* row = xs + static_cast<size_t>(at[s]) * p.width;
#pragma unroll
            for (int w = 0; w < kW; ++w)
                if (in[w]) (at[s] < end ? v[w] : none).store(row + w * step);
        }
    }
}

// y[t] = residual[t] + sum_s weights[t, s] ys[rows[t, s]], over the slots that have an
// expert (what another's place holds is not read).  A thread has kS rows' words on their
// way at once, kW of each row: between the places' arrival and the rows' a CTA asks for
// nothing, so many loads have to follow.  Words of eight bytes, so that many CTAs fit.
// (512 tokens of eight rows of 14336 bytes, 73 MB: words of 16 bytes 16.6 us, of eight
// bytes 16.3, two of them 15.1; 4096 tokens of two rows of 8192 bytes, 134 MB: one
// word of each row 47 us, eight 27.)
template <typename T, int V, int kS, int kW>
__global__ void __launch_bounds__(kMoveThreads) combine_kernel(MoveArgs p) {
    pdl_wait_prerequisites();
    pdl_allow_dependents();
    const int t = blockIdx.x / p.chunks, lane = threadIdx.x & 31;
    const int u = (blockIdx.x - t * p.chunks) * kW * blockDim.x + threadIdx.x;
    const size_t mine = static_cast<size_t>(t) * p.width + static_cast<size_t>(u) * V;
    const int step = blockDim.x * V;  // from one of the thread's words to the next
    const T* ys = static_cast<const T*>(p.in) + static_cast<size_t>(u) * V;
    const size_t slot0 = static_cast<size_t>(t) * p.top_k;
    const unsigned end = static_cast<unsigned>(min(max(__ldg(p.offsets + p.experts), 0), p.routes));
    bool in[kW];
    float sum[kW][V];
    Pack<T, V> r[kW];
#pragma unroll
    for (int w = 0; w < kW; ++w) {
        in[w] = u + w * static_cast<int>(blockDim.x) < p.units;
        r[w].load_if(static_cast<const T*>(p.residual) + mine + w * step, in[w] && p.residual != nullptr);
    }
#pragma unroll
    for (int w = 0; w < kW; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v) sum[w][v] = r[w].get(v);
    for (int s0 = 0; s0 < p.top_k; s0 += kS) {
        // a lane has one of the places and weights
        const bool slot = lane < kS && s0 + lane < p.top_k;
        const int place = slot ? __ldg(p.rows + slot0 + s0 + lane) : -1;
        const float weight = slot && p.weights != nullptr ? __ldg(p.weights + slot0 + s0 + lane) : 1.f;
        int at[kS];
        Pack<T, V> a[kS][kW];
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            at[s] = __shfl_sync(0xFFFFFFFFu, place, s);
            const T* row = ys + static_cast<size_t>(static_cast<unsigned>(at[s])) * p.width;
#pragma unroll
            for (int w = 0; w < kW; ++w) a[s][w].load_if(row + w * step, in[w] && static_cast<unsigned>(at[s]) < end);
        }
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            const float f = __shfl_sync(0xFFFFFFFFu, weight, s);
            if (static_cast<unsigned>(at[s]) >= end) continue;
#pragma unroll
            for (int w = 0; w < kW; ++w)
#pragma unroll
                for (int v = 0; v < V; ++v) sum[w][v] = fmaf(f, a[s][w].get(v), sum[w][v]);
        }
    }
#pragma unroll
    for (int w = 0; w < kW; ++w) {
        if (!in[w]) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) r[w].set(v, sum[w][v]);
        r[w].store(static_cast<T*>(p.out) + mine + w * step);
    }
}

struct BackArgs {
    const void* dy;
    const void* ys;
    const float* weights;
    const int* rows;
    const int* offsets;
    void* dys;
    float* dweights;
    int top_k, routes, experts;
    int width, units;
    int parts;  // CTAs of a cluster that share a row
};

// dys[rows[t, s]] = weights[t, s] dy[t] and dweights[t, s] = <dy[t], ys[rows[t, s]]>:
// dy and ys are read once for both, kW words of a thread from each of kS rows at once.  A
// thread's sums, the warp's, the CTA's and the cluster's are added in that order, whatever
// runs when.  Eight rows' words of 16 bytes leave room for three CTAs of an SM (1024 tokens
// of eight rows of 7168 bf16: three 43.8 us, two 46).  With one or two choices of a token
// two rows at once (4096 tokens of 4096 bf16: eight 54 us, two 30; of 4097 106 and 45), and
// of words of one value two from each of four (1024 tokens of four rows of 4097 bf16: one of
// eight 26 us, so 17; eight of 7169 37 and 35).
template <typename T, int V, int kS, int kW>
__global__ void __launch_bounds__(kMoveThreads, kS == 2 || V <= 2 ? 4 : 3) combine_backward_kernel(BackArgs p) {
    __shared__ float part[kMoveThreads / 32][kS];
    __shared__ float mine[kS];
    pdl_wait_prerequisites();
    pdl_allow_dependents();
    const int t = blockIdx.x / p.parts, rank = blockIdx.x - t * p.parts;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const size_t slot0 = static_cast<size_t>(t) * p.top_k;
    const unsigned end = static_cast<unsigned>(min(max(__ldg(p.offsets + p.experts), 0), p.routes));
    const int u0 = static_cast<int>(static_cast<long long>(p.units) * rank / p.parts);
    const int u1 = static_cast<int>(static_cast<long long>(p.units) * (rank + 1) / p.parts);
    const T* dy = static_cast<const T*>(p.dy) + static_cast<size_t>(t) * p.width;
    const int step = blockDim.x * V;  // from one of the thread's words to the next
    for (int s0 = 0; s0 < p.top_k; s0 += kS) {
        int at[kS];
        float w[kS], dot[kS];
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            at[s] = s0 + s < p.top_k ? __ldg(p.rows + slot0 + s0 + s) : -1;
            w[s] = s0 + s < p.top_k ? __ldg(p.weights + slot0 + s0 + s) : 0.f;
            dot[s] = 0.f;
        }
        for (int u = u0 + threadIdx.x; u < u1; u += kW * blockDim.x) {
            const size_t col = static_cast<size_t>(u) * V;
            Pack<T, V> g[kW], a[kS][kW];
            bool in[kW];
#pragma unroll
            for (int i = 0; i < kW; ++i) {
                in[i] = i == 0 || u + i * static_cast<int>(blockDim.x) < u1;
                if (i == 0) g[i].load(dy + col);
                else g[i].load_if(dy + col + i * step, in[i]);
            }
#pragma unroll
            for (int s = 0; s < kS; ++s) {
                const T* row = static_cast<const T*>(p.ys) + static_cast<size_t>(static_cast<unsigned>(at[s])) * p.width + col;
#pragma unroll
                for (int i = 0; i < kW; ++i) a[s][i].load_if(row + i * step, in[i] && static_cast<unsigned>(at[s]) < end);
            }
#pragma unroll
            for (int s = 0; s < kS; ++s) {
                if (static_cast<unsigned>(at[s]) >= static_cast<unsigned>(p.routes)) continue;
                T* to = static_cast<T*>(p.dys) + static_cast<size_t>(at[s]) * p.width + col;
#pragma unroll
                for (int i = 0; i < kW; ++i) {
                    Pack<T, V> d;
                    if (static_cast<unsigned>(at[s]) < end) {
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            dot[s] = fmaf(g[i].get(v), a[s][i].get(v), dot[s]);
                            d.set(v, w[s] * g[i].get(v));
                        }
                    }
                    if (in[i]) d.store(to + i * step);
                }
            }
        }
#pragma unroll
        for (int s = 0; s < kS; ++s) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) dot[s] += __shfl_xor_sync(0xFFFFFFFFu, dot[s], d);
            if (lane == 0) part[warp][s] = dot[s];
        }
        __syncthreads();
        float sum = 0.f;
        if (threadIdx.x < kS) {
            for (int i = 0; i < warps; ++i) sum += part[i][threadIdx.x];
            mine[threadIdx.x] = sum;
        }
        if (p.parts > 1) {
            cluster_arrive();
            cluster_wait();
            if (rank == 0 && threadIdx.x < kS) {
                sum = 0.f;
                for (int c = 0; c < p.parts; ++c)
                    sum += __uint_as_float(load_cluster_u32(smem_u32(mine + threadIdx.x), c));
            }
        }
        if (rank == 0 && threadIdx.x < kS && s0 + static_cast<int>(threadIdx.x) < p.top_k)
            p.dweights[slot0 + s0 + threadIdx.x] = sum;
        if (p.parts > 1) {  // the sums are read before they change or their CTA leaves
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
    }
}

// ---- launches --------------------------------------------------------------------

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

// The widest word (in bytes, up to 16) that rows of `row_bytes` and all the pointers
// (ORed) are multiples of.
int word_bytes(size_t row_bytes, uintptr_t pointers) {
    const uintptr_t low = row_bytes | pointers | 16;
    return static_cast<int>(low & (~low + 1));
}

// Calls f with the number of values in a word of `bytes`.
template <typename T, typename F>
cudaError_t with_values(int bytes, F&& f) {
    switch (bytes) {
        case 16: return f(std::integral_constant<int, 16 / sizeof(T)>{});
        case 8: return f(std::integral_constant<int, 8 / sizeof(T)>{});
        case 4: return f(std::integral_constant<int, 4 / sizeof(T)>{});
        case 2:
            if constexpr (sizeof(T) == 2) return f(std::integral_constant<int, 1>{});
    }
    return cudaErrorInvalidValue;
}

template <typename T, bool kCombine>
cudaError_t launch_move(const MoeMoveArgs& a, cudaStream_t stream) {
    MoveArgs p = {};
    p.in = a.in;
    p.residual = a.residual;
    p.weights = a.weights;
    p.rows = a.rows;
    p.offsets = a.offsets;
    p.out = a.out;
    p.top_k = a.top_k;
    p.routes = a.n_tokens * a.top_k;
    p.experts = a.n_experts;
    p.width = a.width;
    const int bytes = std::min(kCombine ? 8 : 16,
                               word_bytes(static_cast<size_t>(a.width) * sizeof(T),
                                          reinterpret_cast<uintptr_t>(a.in) | reinterpret_cast<uintptr_t>(a.out) |
                                              reinterpret_cast<uintptr_t>(a.residual)));
    return with_values<T>(bytes, [&](auto values) {
        constexpr int V = decltype(values)::value;
        p.units = a.width / V;
        // a row's words in equal chunks of `each` a thread, whole warps each
        auto go = [&](void (*kernel)(MoveArgs), int each) {
            p.chunks = (p.units + each * kMoveThreads - 1) / (each * kMoveThreads);
            const int chunk = (p.units + p.chunks - 1) / p.chunks;
            const int threads = ((chunk + each - 1) / each + 31) & ~31;
            return launch_pdl(kernel, dim3(static_cast<unsigned>(a.n_tokens) * p.chunks), threads, 0, 1, stream, p);
        };
        if constexpr (kCombine) {
            if constexpr (V * sizeof(T) > 8) return cudaErrorInvalidValue;  // (no such words here)
            else if (a.top_k <= 2) return go(combine_kernel<T, V, 2, 8>, 8);
            else return go(combine_kernel<T, V, kSlots, V * sizeof(T) == 8 ? 2 : 4>, V * sizeof(T) == 8 ? 2 : 4);
        } else {
            constexpr int kW = 16 / (V * sizeof(T));
            return go(sort_kernel<T, V, kW>, kW);
        }
    });
}

template <typename T>
cudaError_t launch_back(const MoeBackArgs& a, cudaStream_t stream) {
    BackArgs p = {};
    p.dy = a.dy;
    p.ys = a.ys;
    p.weights = a.weights;
    p.rows = a.rows;
    p.offsets = a.offsets;
    p.dys = a.dys;
    p.dweights = a.dweights;
    p.top_k = a.top_k;
    p.routes = a.n_tokens * a.top_k;
    p.experts = a.n_experts;
    p.width = a.width;
    const int bytes = word_bytes(static_cast<size_t>(a.width) * sizeof(T),
                                 reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.ys) |
                                     reinterpret_cast<uintptr_t>(a.dys));
    return with_values<T>(bytes, [&](auto values) {
        constexpr int V = decltype(values)::value;
        p.units = a.width / V;
        auto go = [&](void (*kernel)(BackArgs), int each) {
            // (`each` words of a thread at once)
            const int threads = std::min(kMoveThreads, ((p.units + each - 1) / each + 31) & ~31);
            p.parts = 1;
            while (p.parts < kRouteMaxCtas && a.n_tokens * p.parts < 2 * a.sm_count &&
                   2 * p.parts * threads * each <= p.units)
                p.parts *= 2;
            const dim3 grid(static_cast<unsigned>(a.n_tokens) * p.parts);
            return launch_pdl(kernel, grid, threads, 0, p.parts, stream, p);
        };
        constexpr int kW = std::min(4, static_cast<int>(32 / (V * sizeof(T))));
        if (a.top_k <= 2) return go(combine_backward_kernel<T, V, 2, kW>, kW);
        if constexpr (V == 1) return go(combine_backward_kernel<T, V, 4, 2>, 2);
        else return go(combine_backward_kernel<T, V, kSlots, 1>, 1);
    });
}

}  // namespace

cudaError_t launch_moe_route(const MoeRouteArgs& a, cudaStream_t stream) {
    const int bins = a.n_experts + 1;
    RouteArgs p = {};
    p.ids = a.ids;
    p.rows = a.rows;
    p.order = a.order;
    p.offsets = a.offsets;
    p.bad_ids = a.bad_ids;
    p.routes = a.n_tokens * a.top_k;
    p.experts = a.n_experts;
    while (p.experts >> p.bits) ++p.bits;
    // a warp takes 32 choices, and up to kRouteEach before further CTAs share them: the
    // walks over warps and CTAs cost as much as the steps that they save
    const int most = bins <= kRouteFewBins ? kRouteWarps : kRouteWarpsMany;
    const int warps = std::min(most, (p.routes + 31) / 32);
    int ctas = 1;
    while (ctas < kRouteMaxCtas && ctas * warps * kRouteEach < p.routes) ctas *= 2;
    p.each = ((p.routes + ctas * warps - 1) / (ctas * warps) + 31) & ~31;
    const size_t smem = (static_cast<size_t>(warps + 2) * bins + 1) * 4;
    static std::atomic<bool> attr_done[64] = {};  // (set by any thread; setting twice does no harm)
    if (a.device < 0 || a.device >= 64) return cudaErrorInvalidDevice;
    if (smem > 48 * 1024 && !attr_done[a.device].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute(route_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
        attr_done[a.device].store(true, std::memory_order_release);
    }
    return launch_pdl(route_kernel, dim3(ctas), 32 * warps, smem, ctas, stream, p);
}

cudaError_t launch_moe_sort(const MoeMoveArgs& a, cudaStream_t stream) {
    return a.bf16 ? launch_move<__nv_bfloat16, false>(a, stream) : launch_move<float, false>(a, stream);
}

cudaError_t launch_moe_combine(const MoeMoveArgs& a, cudaStream_t stream) {
    return a.bf16 ? launch_move<__nv_bfloat16, true>(a, stream) : launch_move<float, true>(a, stream);
}

cudaError_t launch_moe_combine_backward(const MoeBackArgs& a, cudaStream_t stream) {
    return a.bf16 ? launch_back<__nv_bfloat16>(a, stream) : launch_back<float>(a, stream);
}

}  // namespace q2k
