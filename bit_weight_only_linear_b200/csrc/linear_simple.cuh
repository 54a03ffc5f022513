// Fused linear and expert-grouped linear, direct form: one warp per (output channel, up to 8
// rows), the lanes striding over the packed words, fp32 products and sums.  Bound by the
// CUDA cores' multiply-adds.
#pragma once

#include "common.cuh"
#include "epilogue.cuh"

namespace awq {

constexpr int kSimpleRows = 8;
constexpr int kSimpleThreads = 256;

// Row range of expert e, clamped into 0..R whatever the table holds.
__device__ __forceinline__ int2 expert_range(const int32_t* offsets, int e, int R) {
    const int b = min(max(__ldg(offsets + e), 0), R);
    return make_int2(b, min(max(__ldg(offsets + e + 1), b), R));
}

__global__ void __launch_bounds__(kSimpleThreads)
linear_simple_kernel(const uint16_t* __restrict__ X, int T, long long ldx, const int32_t* __restrict__ rows, int R,
                     const int32_t* __restrict__ offsets, int E, const uint32_t* __restrict__ qweight,
                     const uint16_t* __restrict__ scales, const uint32_t* __restrict__ qzeros, int N, int K, int G,
                     Epilogue ep) {
    const int lane = threadIdx.x & 31;
    const int F = ep.gated ? N / 2 : N;
    const int f = blockIdx.x * (kSimpleThreads / 32) + (threadIdx.x >> 5);
    // tile blockIdx.y of 8 rows: the experts' ranges, each in tiles of its own
    int e = 0, r0 = blockIdx.y * kSimpleRows, r1 = R;
    if (offsets) {
        int tile = blockIdx.y;
        for (; e < E; ++e) {
            const int2 g = expert_range(offsets, e, R);
            const int tiles = (g.y - g.x + kSimpleRows - 1) / kSimpleRows;
            if (tile < tiles) {
                r0 = g.x + tile * kSimpleRows;
                r1 = g.y;
                break;
            }
            tile -= tiles;
        }
        if (e == E) return;
    }
    if (f >= F) return;
    const int nr = min(kSimpleRows, r1 - r0);
    const int ng = K / G, nzw = (ng + 7) / 8, kw = K / 8;
    const uint16_t* x[kSimpleRows];
    bool live[kSimpleRows];
    for (int i = 0; i < kSimpleRows; ++i) {
        const int src = i < nr ? (rows ? rows[r0 + i] : r0 + i) : -1;
        live[i] = src >= 0 && src < T;
        x[i] = X + (live[i] ? src : 0) * ldx;
    }
    float v[2][kSimpleRows];
    for (int h = 0; h < (ep.gated ? 2 : 1); ++h) {
        const size_t n = (size_t)e * N + h * F + f;
        float acc[kSimpleRows] = {};
        for (int w = lane; w < kw; w += 32) {
            const uint32_t q = qweight[n * kw + w];
            const int g = w * 8 / G;
            const float s = h2f(scales[n * ng + g]);
            const int z = qzeros ? (qzeros[n * nzw + g / 8] >> (4 * (g & 7))) & 15 : 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int nib = (j >> 1) + 4 * (j & 1);      // codes k, k+1: the same nibble of the word's halves
                const float d = (float)((int)((q >> (4 * nib)) & 15u) - z) * s;
#pragma unroll
                for (int i = 0; i < kSimpleRows; ++i)
                    if (live[i]) acc[i] = fmaf(d, h2f(x[i][w * 8 + j]), acc[i]);
            }
        }
        for (int i = 0; i < kSimpleRows; ++i) {
            for (int o = 16; o; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
            v[h][i] = acc[i] + (ep.bias ? h2f(ep.bias[n]) : 0.0f);
        }
    }
    if (lane == 0)
        for (int i = 0; i < nr; ++i) {
            float y = apply_act(v[0][i], ep.act);
            if (ep.gated) y *= v[1][i];
            if (ep.residual) y += h2f(ep.residual[(r0 + i) * ep.ldr + f]);
            ep.Y[(r0 + i) * ep.ldy + f] = f2h_rn(y);
        }
}

inline awq_status launch_linear_simple(const uint16_t* X, int T, long long ldx, const int32_t* rows, int R,
                                       const int32_t* offsets, int E, const uint32_t* qweight, const uint16_t* scales,
                                       const uint32_t* qzeros, int N, int K, int G, const Epilogue& ep,
                                       cudaStream_t st) {
    const long long tiles = offsets ? R / kSimpleRows + (R < E ? R : E) : ceil_div(R, kSimpleRows);
    const dim3 grid(ceil_div(ep.gated ? N / 2 : N, kSimpleThreads / 32), (unsigned)tiles);
    if (tiles > 65535) return AWQ_ERR_UNSUPPORTED;
    linear_simple_kernel<<<grid, kSimpleThreads, 0, st>>>(X, T, ldx, rows, R, offsets, E, qweight, scales, qzeros, N,
                                                          K, G, ep);
    return cudaGetLastError() == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

}  // namespace awq
