// Expert routing and combination of a mixture-of-experts layer around the grouped linear.
//
// Routing.  Per token: the top_k largest logits (ties to the lower expert), their weights,
// and the stable order of the chosen (token, expert) slots by expert: offsets[e] is the first
// row of expert e, rows[p] the token of row p, positions[t][j] the row of slot j of token t.
//   * A warp per token holds the logits in registers (expert = 32 s + lane) as order-preserving
//     integers; each of the top_k rounds is two warp reductions (largest key, then lowest index).
//   * Stable counting sort without atomics on counters: a token takes an expert at most once, so
//     inside a chunk of 32 tokens the rank of a slot is the population count of the lower tokens'
//     bits in the expert's 32-bit mask (the masks are built by atomicOr, whose result does not
//     depend on order).  Blocks take contiguous ranges of tokens and publish their counts; the
//     second kernel adds the counts of the blocks before its own.  One block needs no second
//     kernel.
// Bound: a few launches' latency for decode; for a long prefill the top_k rounds (issue).
//
// Combination.  out[t] = residual[t] + sum_j w[t][j] Y[positions[t][j]], fp32 sums in slot order,
// one rounding: bound by reading the T top_k rows once.
#pragma once

#include "common.cuh"
#include "gemv_launch.cuh"

namespace awq {

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 32;
constexpr int kRouteChunk = 32;         // tokens ranked at a time (one bit each)
constexpr int kRouteThreads = 1024;     // 32 warps: one token each per chunk
// Tokens that one block takes alone in a single launch.
constexpr int kRouteSingle = 256;

struct RouteArgs {
    const void* logits;
    long long ld;
    int half;              // fp16 logits (else fp32)
    int T, E, k, sigmoid, renorm;
    float* weights;
    int32_t *experts, *offsets, *rows, *positions;
    uint16_t* counts;      // [blocks][E]: slots of each block
    int per_block;         // tokens per block (a multiple of kRouteChunk)
    int blocks;
};

// Order-preserving key of a logit: larger logits have larger keys; 0 = masked (-inf or NaN).
__device__ __forceinline__ uint32_t logit_key(float l) {
    if (!(l > -INFINITY)) return 0u;                 // -inf, NaN
    const uint32_t u = __float_as_uint(l + 0.0f);    // -0 -> +0: they tie
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// Exclusive prefix sum of cnt[0..E) into base[0..E], by the whole block (E <= kRouteThreads).
__device__ __forceinline__ void block_prefix(const int* cnt, int* base, int E, int* warp_sums) {
    const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
    const int v = i < E ? cnt[i] : 0;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    const int before = (warp ? warp_sums[warp - 1] : 0) + x - v;
    if (i < E) base[i] = before;
    if (i == E - 1) base[E] = before + v;
    __syncthreads();
}

// NS registers of keys per lane: up to 32 NS experts.  positions[] receives the slot's rank among
// its block's rows of the expert (the final row when there is one block).
template <int NS>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(RouteArgs a) {
    __shared__ int run[kRouteMaxExperts];            // rows of each expert before the chunk
    __shared__ uint32_t mask[kRouteMaxExperts];      // tokens of the chunk that chose it
    __shared__ int base[kRouteMaxExperts + 1];
    __shared__ int warp_sums[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) run[e] = 0, mask[e] = 0;
    __syncthreads();
    const int t_begin = blockIdx.x * a.per_block;
    const int t_end = min(a.T, t_begin + a.per_block);
    for (int t0 = t_begin; t0 < t_end; t0 += kRouteChunk) {
        const int t = t0 + warp;
        int chosen = -1;
        if (t < t_end) {
            uint32_t key[NS];
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int e = s * 32 + lane;
                key[s] = 0;
                if (e < a.E)
                    key[s] = logit_key(a.half ? h2f(static_cast<const uint16_t*>(a.logits)[t * a.ld + e])
                                              : static_cast<const float*>(a.logits)[t * a.ld + e]);
            }
            // softmax over every expert that is not masked: exp(l - top), +inf as the largest finite value
            uint32_t top = 0;
#pragma unroll
            for (int s = 0; s < NS; ++s) top = max(top, key[s]);
            top = __reduce_max_sync(0xffffffffu, top);
            const float lmax = top ? fminf(key_logit(top), 3.402823466e38f) : 0.0f;
            float total = 0.0f;
            if (!a.sigmoid && !a.renorm) {
#pragma unroll
                for (int s = 0; s < NS; ++s)
                    if (key[s]) total += expf(fminf(key_logit(key[s]), 3.402823466e38f) - lmax);
#pragma unroll
                for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
            }
            uint32_t chosen_key = 0;
            for (int j = 0; j < a.k; ++j) {
                uint32_t bk = 0;
                int be = 0x7fffffff;
#pragma unroll
                for (int s = 0; s < NS; ++s)
                    if (key[s] > bk) bk = key[s], be = s * 32 + lane;
                const uint32_t wk = __reduce_max_sync(0xffffffffu, bk);
                if (wk == 0) break;                                   // only masked experts are left
                const int we = (int)__reduce_min_sync(0xffffffffu, bk == wk ? (uint32_t)be : 0x7fffffffu);
#pragma unroll
                for (int s = 0; s < NS; ++s)
                    if (we == s * 32 + lane) key[s] = 0;
                if (lane == j) chosen = we, chosen_key = wk;
            }
            float w = 0.0f;
            if (chosen >= 0) {
                const float l = fminf(key_logit(chosen_key), 3.402823466e38f);
                w = a.sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - lmax);
                if (!a.sigmoid && !a.renorm) w /= total;
            }
            if (a.renorm) {
                float sum = w;
#pragma unroll
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                w = sum > 0.0f ? w / sum : 0.0f;
            }
            if (lane < a.k) {
                a.weights[(size_t)t * a.k + lane] = w;
                a.experts[(size_t)t * a.k + lane] = chosen;
            }
            if (chosen >= 0) atomicOr(&mask[chosen], 1u << warp);
        }
        __syncthreads();
        if (t < t_end && lane < a.k)
            a.positions[(size_t)t * a.k + lane] =
                chosen < 0 ? -1 : run[chosen] + __popc(mask[chosen] & ((1u << warp) - 1u));
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += kRouteThreads) {
            run[e] += __popc(mask[e]);
            mask[e] = 0;
        }
        __syncthreads();
    }
    if (a.blocks > 1) {
        for (int e = threadIdx.x; e < a.E; e += kRouteThreads)
            a.counts[(size_t)blockIdx.x * a.E + e] = (uint16_t)run[e];
        return;
    }
    // one block: the order is complete
    block_prefix(run, base, a.E, warp_sums);
    for (int e = threadIdx.x; e <= a.E; e += kRouteThreads) a.offsets[e] = base[e];
    const int slots = a.T * a.k;
    for (int i = threadIdx.x; i < slots; i += kRouteThreads) {
        const int e = a.experts[i];
        if (e < 0) continue;
        const int p = base[e] + a.positions[i];
        a.positions[i] = p;
        a.rows[p] = i / a.k;
    }
    for (int p = base[a.E] + threadIdx.x; p < slots; p += kRouteThreads) a.rows[p] = -1;
}

// Second step: every block adds the counts of the blocks before it and turns its slots' ranks
// into rows.
__global__ void __launch_bounds__(kRouteThreads) route_order_kernel(RouteArgs a) {
    __shared__ int total[kRouteMaxExperts], before[kRouteMaxExperts];
    __shared__ int base[kRouteMaxExperts + 1];
    __shared__ int warp_sums[32];
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) total[e] = before[e] = 0;
    __syncthreads();
    // thread (part, expert): the counts of every parts-th block (integer sums: order-free)
    const int parts = max(1, kRouteThreads / a.E);
    const int e0 = threadIdx.x % a.E, part = threadIdx.x / a.E;
    if (part < parts) {
        int tot = 0, bef = 0;
#pragma unroll 8
        for (int b = part; b < a.blocks; b += parts) {
            const int c = a.counts[(size_t)b * a.E + e0];
            tot += c;
            bef += b < (int)blockIdx.x ? c : 0;
        }
        atomicAdd(&total[e0], tot);
        atomicAdd(&before[e0], bef);
    }
    __syncthreads();
    block_prefix(total, base, a.E, warp_sums);
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= a.E; e += kRouteThreads) a.offsets[e] = base[e];
    const size_t s_begin = (size_t)blockIdx.x * a.per_block * a.k;
    const size_t s_end = min((size_t)a.T, (size_t)(blockIdx.x + 1) * a.per_block) * a.k;
    for (size_t i = s_begin + threadIdx.x; i < s_end; i += kRouteThreads) {
        const int e = a.experts[i];
        if (e >= 0) {
            const int p = base[e] + before[e] + a.positions[i];
            a.positions[i] = p;
            a.rows[p] = (int)(i / a.k);
        }
        if (i >= (size_t)base[a.E]) a.rows[i] = -1;      // behind the last expert's rows
    }
}

inline int route_blocks(int T, int sms, int& per_block) {
    if (T <= kRouteSingle) {
        per_block = ceil_div(T, kRouteChunk) * kRouteChunk;
        return 1;
    }
    per_block = ceil_div(ceil_div(T, sms), kRouteChunk) * kRouteChunk;
    return ceil_div(T, per_block);
}

inline size_t route_workspace_bytes(int T, int E, int sms) {
    if (T <= 0 || E <= 0) return 0;
    int per = 0;
    const int blocks = route_blocks(T, sms, per);
    return blocks > 1 ? align256((size_t)blocks * E * 2) : 0;
}

inline awq_status launch_route(RouteArgs a, cudaStream_t st) {
    const unsigned g = (unsigned)a.blocks;
    if (a.E <= 32) route_kernel<1><<<g, kRouteThreads, 0, st>>>(a);
    else if (a.E <= 64) route_kernel<2><<<g, kRouteThreads, 0, st>>>(a);
    else if (a.E <= 128) route_kernel<4><<<g, kRouteThreads, 0, st>>>(a);
    else if (a.E <= 256) route_kernel<8><<<g, kRouteThreads, 0, st>>>(a);
    else if (a.E <= 512) route_kernel<16><<<g, kRouteThreads, 0, st>>>(a);
    else route_kernel<32><<<g, kRouteThreads, 0, st>>>(a);
    if (a.blocks > 1) route_order_kernel<<<g, kRouteThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

// ---------------------------------------------------------------------------

constexpr int kCombineThreads = 128;

template <int V> struct HalfVec;
template <> struct HalfVec<8> { using T = uint4; };
template <> struct HalfVec<2> { using T = uint32_t; };
template <> struct HalfVec<1> { using T = uint16_t; };

// V columns per thread and load (V halves aligned to their size in every row).
template <int V>
__global__ void __launch_bounds__(kCombineThreads)
combine_kernel(const uint16_t* __restrict__ Y, int R, long long ldy, const float* __restrict__ weights,
               const int32_t* __restrict__ positions, int k, int N, const uint16_t* residual, long long ldr,
               uint16_t* out, long long ldo) {
    using Vec = typename HalfVec<V>::T;
    const size_t t = blockIdx.x;
    const int n = (blockIdx.y * kCombineThreads + threadIdx.x) * V;
    if (n >= N) return;
    float acc[V] = {};
    constexpr int kAhead = 4;                        // rows in flight per thread
    for (int j0 = 0; j0 < k; j0 += kAhead) {
        Vec v[kAhead];
        float w[kAhead];
        bool live[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int p = j0 + i < k ? __ldg(positions + t * k + j0 + i) : -1;
            live[i] = p >= 0 && p < R;
            if (live[i]) {
                w[i] = __ldg(weights + t * k + j0 + i);
                v[i] = *reinterpret_cast<const Vec*>(Y + p * ldy + n);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (live[i]) {
                const uint16_t* h = reinterpret_cast<const uint16_t*>(&v[i]);
#pragma unroll
                for (int c = 0; c < V; ++c) acc[c] = fmaf(w[i], h2f(h[c]), acc[c]);
            }
    }
    if (residual) {
        const Vec r = *reinterpret_cast<const Vec*>(residual + t * ldr + n);
        const uint16_t* h = reinterpret_cast<const uint16_t*>(&r);
#pragma unroll
        for (int c = 0; c < V; ++c) acc[c] += h2f(h[c]);
    }
    Vec o;
    uint16_t* h = reinterpret_cast<uint16_t*>(&o);
#pragma unroll
    for (int c = 0; c < V; ++c) h[c] = f2h_rn(acc[c]);
    *reinterpret_cast<Vec*>(out + t * ldo + n) = o;
}

inline awq_status launch_combine(const uint16_t* Y, int R, long long ldy, const float* weights,
                                 const int32_t* positions, int T, int k, int N, const uint16_t* residual,
                                 long long ldr, uint16_t* out, long long ldo, cudaStream_t st) {
    // widest load that every row's start allows
    const uintptr_t a = reinterpret_cast<uintptr_t>(Y) | reinterpret_cast<uintptr_t>(out) |
                        reinterpret_cast<uintptr_t>(residual) |
                        (uintptr_t)(2 * (ldy | ldo | (residual ? ldr : 0) | (long long)N));
    auto grid = [&](int V) { return dim3((unsigned)T, ceil_div(N, kCombineThreads * V)); };
#define AWQ_COMBINE(V) \
    combine_kernel<V><<<grid(V), kCombineThreads, 0, st>>>(Y, R, ldy, weights, positions, k, N, residual, ldr, out, ldo)
    if ((a & 15) == 0) AWQ_COMBINE(8);
    else if ((a & 3) == 0) AWQ_COMBINE(2);
    else AWQ_COMBINE(1);
#undef AWQ_COMBINE
    return cudaGetLastError() == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

}  // namespace awq
