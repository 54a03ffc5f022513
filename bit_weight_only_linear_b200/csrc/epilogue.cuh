// Epilogue of the fused linears: bias, activation, the gated product and the residual, on
// fp32 accumulators with one fp16 rounding at the store.
//
//   plain  y = act(acc + b) + r
//   gated  y = act(acc_f + b_f) * (acc_{F+f} + b_{F+f}) + r       (N = 2F weight rows)
//
// The activations are evaluated in fp32 with CUDA's exp, erfc and approximate division: fp16
// keeps 11 bits, so their errors of a few fp32 units vanish in the one rounding.
#pragma once

#include "common.cuh"

namespace awq {

struct Epilogue {
    const uint16_t* bias;       // [N] (grouped: [E][N]) or NULL
    const uint16_t* residual;   // [M][ldr] or NULL
    long long ldr;
    uint16_t* Y;                // [M][ldy]
    long long ldy;
    int act;                    // awq_activation
    int gated;
};

// Out of line: the epilogues unroll over 16 accumulators, and 16 inlined copies of erfc made their
// code so long that fetching it cost more than running it (20 us for one 256 x 192 tile).
__device__ __noinline__ float act_gelu(float v) {
    return 0.5f * v * erfcf(v * -0.70710678f);      // erfc: no cancellation at v << 0
}

__device__ __forceinline__ float act_sigmoid_form(float v, float w) { return __fdividef(v, 1.0f + __expf(-w)); }

// v[i] <- act(v[i]); the branch on the activation is outside the loop over the values.
template <int C>
__device__ __forceinline__ void apply_act(float (&v)[C], int act) {
    if (act == AWQ_ACT_NONE) return;
    if (act == AWQ_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];          // keeps NaN
    } else if (act == AWQ_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = act_sigmoid_form(v[i], v[i]);
    } else if (act == AWQ_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = act_gelu(v[i]);
    } else {
        // 0.5 v (1 + tanh u) = v / (1 + exp(-2u))
#pragma unroll
        for (int i = 0; i < C; ++i)
            v[i] = act_sigmoid_form(v[i], 1.59576912f * (v[i] + 0.044715f * v[i] * v[i] * v[i]));
    }
}

}  // namespace awq
