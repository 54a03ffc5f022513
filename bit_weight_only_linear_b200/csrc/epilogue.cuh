// Epilogue of the fused linears: bias, activation, the gated product and the residual, on
// fp32 accumulators with one fp16 rounding at the store.
//
//   plain  y = act(acc + b) + r
//   gated  y = act(acc_f + b_f) * (acc_{F+f} + b_{F+f}) + r       (N = 2F weight rows)
//
// The activations are evaluated in fp32 with CUDA's exp and erfc: fp16 keeps 11 bits,
// so their errors of a few fp32 units vanish in the one rounding.
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

__device__ __forceinline__ float apply_act(float v, int act) {
    switch (act) {
        case AWQ_ACT_RELU: return v < 0.0f ? 0.0f : v;            // keeps NaN
        case AWQ_ACT_SILU: return v / (1.0f + __expf(-v));
        case AWQ_ACT_GELU: return 0.5f * v * erfcf(v * -0.70710678f);   // erfc: no cancellation at v << 0
        case AWQ_ACT_GELU_TANH: {
            const float u = 0.79788456f * (v + 0.044715f * v * v * v);
            return v / (1.0f + __expf(-2.0f * u));                // 0.5 v (1 + tanh u)
        }
        default: return v;
    }
}

}  // namespace awq
