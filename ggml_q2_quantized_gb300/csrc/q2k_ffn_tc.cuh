// What the host side of the feed-forward operators' tensor-core kernel shares with its
// instantiations (one file for each mode, so that they compile side by side).
#pragma once

#include "q2k_ffn.cuh"
#include "q2k_ffn_plan.h"
#include "q2k_internal.h"
#include "q2k_tc.cuh"

namespace q2k {

// kLinear: one matrix, with bias, activation and residual; kBackward: one matrix or two.
enum class Tc { kGated, kLora, kLinear, kBackward };

struct TcArgs {
    const uint8_t* xa;   // bf16 image of the tokens, or null: they come by the token maps
    const uint8_t* w0;   // Wg, or W
    const uint8_t* w1;   // Wu
    int groups;          // fours of weight rows that the maps cover, 0: none
    int M, N, K;         // N, K: the weight matrices' rows and columns
    int quads;           // the product's K in blocks (backward: 256 weight rows)
    int half_stages;     // backward: 64-row stages of Wg
    int tiles, row_units;  // tiles, row tiles (256 tokens: pairs of them) first
    int whole;           // tiles [0, whole) go to the workers in turn, the rest is cut
    int parts;           // CTAs (pairs) of a cluster that divide K (then one tile each)
    float* partial;      // sums of a cut tile's runs, two slots per CTA
    unsigned int* counts;  // per cut tile and CTA of a worker: runs finished (zeroed)
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
    // one matrix (y as above)
    const float* bias;   // [n_experts][N], or null
    const void* residual;
    void* z;             // x W^T + bias, or null
    // tokens in segments (kSeg), each with matrices of its own: the token tiles and how
    // many
    const int4* table;
    const int* table_count;
};

// Makes the address of a file's error word (a __device__ variable) known to
// read_and_clear_ffn_error; true.
bool add_tc_error_word(const void* symbol);

// Launch the kernel: results of type T; with kSeg tokens in segments.
//   workspace    the plan's sums and counts (zeroed)
//   x0, x1       bf16 token matrices [M, x_cols] with rows `x_pitch` apart (x1: backward,
//                du), or null with a.xa an image
//   experts      matrices, one after another (kSeg)
template <Tc kMode, typename T, bool kSeg>
cudaError_t launch_tc(TcArgs a, const Plan& plan, uint8_t* workspace, const void* x0, const void* x1,
                      int x_cols, int x_pitch, int device, cudaStream_t stream, int experts);

namespace tc {

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace tc

}  // namespace q2k
