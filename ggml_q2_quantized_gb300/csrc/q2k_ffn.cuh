// Device helpers of the feed-forward operators: 32-bit arithmetic on f32 or
// bf16 activations and the two activations with their slopes.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace q2k {

constexpr int kActSilu = 0;
constexpr int kActGelu = 1;  // the tanh form
constexpr int kActNone = 2;

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// D (+)= A B for 16 rows, 16 K and 8 columns: bf16 operands, f32 sums.
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The smaller of two pairs of bf16; of a NaN and a number, the number.
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// act(g) = g p and act'(g) = p + g (1 - p) p z'(g), with p = 1 / (1 + e^-z):
//   silu  z = g                                     z' = 1
//   gelu  z = 2 sqrt(2/pi) (g + 0.044715 g^3)       z' = 2 sqrt(2/pi) (1 + 3 * 0.044715 g^2)
// ((1 + tanh y) / 2 = 1 / (1 + e^-2y), so the tanh form is a logistic too.)
// For the tanh form g is held to |g| <= 30 inside z and z', where p is 0 or 1
// to f32 already: no power of g overflows, and 0 * inf does not arise.
// kFast: e^-z and the quotient by the short instruction sequences, a few units
// in the last place of f32 each; for results that are rounded to bf16.
template <bool kFast>
__device__ __forceinline__ void act_logistic(float g, int act, float& p, float& dz) {
    constexpr float kC = 1.5957691216057308f;  // 2 sqrt(2/pi)
    float z = g;
    dz = 1.0f;
    if (act == kActGelu) {
        const float c = fminf(fmaxf(g, -30.0f), 30.0f);
        z = kC * (c + 0.044715f * c * c * c);
        dz = kC * (1.0f + 3.0f * 0.044715f * c * c);
    }
    p = kFast ? __fdividef(1.0f, 1.0f + __expf(-z)) : 1.0f / (1.0f + expf(-z));
}
template <bool kFast>
__device__ __forceinline__ float act_value(float g, int act) {
    float p, dz;
    act_logistic<kFast>(g, act, p, dz);
    return g * p;
}
template <bool kFast>
__device__ __forceinline__ void act_value_slope(float g, int act, float& value, float& slope) {
    float p, dz;
    act_logistic<kFast>(g, act, p, dz);
    value = g * p;
    slope = p + g * (1.0f - p) * p * dz;
}

}  // namespace q2k
