// Expert routing and combination of a mixture-of-experts layer around the grouped linear.
//
// Routing.  Per token: the top_k largest logits (ties to the lower expert), their weights,
// and the stable order of the chosen (token, expert) slots by expert: offsets[e] is the first
// row of expert e, rows[p] the token of row p, positions[t][j] the row of slot j of token t.
//   * A warp per token holds the logits in registers (expert = 32 s + lane) as order-preserving
//     integers.  Each lane sorts its few, so that a round of the top_k looks at the lanes' heads only:
//     two warp reductions (largest key, then lowest expert) and a pop in one lane.
//   * Stable counting sort without atomics on counters: a token takes an expert at most once, so
//     inside a pass of 128 tokens the rank of a slot is the population count of the lower tokens'
//     bits in the expert's mask (the masks are built by atomicOr, whose result does not depend on
//     order).  Blocks take contiguous ranges of tokens and publish their counts; the second kernel
//     adds the counts of the blocks before its own.  One block needs no second kernel.
// Bound: a launch's latency for decode (8 tokens, 8 experts: 3.7 us); for a long prefill the latency of the
// walks and of the second launch (16384 tokens, top 8 of 128, fp16: 15 us).
//
// Combination.  out[t] = residual[t] + sum_j w[t][j] Y[positions[t][j]], fp32 sums in slot order,
// one rounding: bound by reading the T top_k rows once (8192 tokens x 8 x 4096: 103 us = 6.46 TB/s, 0.99 of the
// measured copy rate).
#pragma once

#include <algorithm>

#include "common.cuh"
#include "gemv_launch.cuh"
#include "linear_common.cuh"

namespace awq {

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 32;
constexpr int kRouteThreads = 1024;     // 32 warps
constexpr int kRouteWords = 4;          // tokens of a warp in a pass; mask words of an expert
constexpr int kRoutePass = 32 * kRouteWords;
constexpr int kRouteSingle = 32;        // tokens that one block takes alone in a single launch

struct RouteArgs {
    const void* logits;
    long long ld;
    int half;              // fp16 logits (else fp32)
    int T, E, k, sigmoid, renorm;
    float* weights;
    int32_t *experts, *offsets, *rows, *positions;
    uint16_t* counts;      // [blocks][E]: slots of each block
    int per_block;         // tokens per block (a multiple of 32)
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

// Sigmoid score e^l / (1 + e^l), times e^-shift; no exponential overflows.  Scores that are divided by their
// sum are taken relative to the token's largest logit where that is negative (shift = min(top, 0)): below -87 the
// scores themselves are denormals, below -104 nothing in fp32, while their shares are ordinary numbers.  A
// logit from kLowestScored down scores 0, so that a lowest finite value written as a mask gives no weight.
constexpr float kLowestScored = -700.0f;

__device__ __forceinline__ float sigmoid_score(float l, float shift) {
    return l > kLowestScored ? expf(fminf(l, 0.0f) - shift) / (1.0f + expf(-fabsf(l))) : 0.0f;
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

// Sorts a lane's keys falling, equal keys in rising slot order (adjacent exchanges only: stable).
template <int NS>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[NS], int (&slot)[NS]) {
#pragma unroll
    for (int n = NS - 1; n > 0; --n)
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const bool swap = key[i + 1] > key[i];
            const uint32_t k0 = swap ? key[i + 1] : key[i], k1 = swap ? key[i] : key[i + 1];
            const int s0 = swap ? slot[i + 1] : slot[i], s1 = swap ? slot[i] : slot[i + 1];
            key[i] = k0, key[i + 1] = k1;
            slot[i] = s0, slot[i + 1] = s1;
        }
}

// NS registers of keys per lane: up to 32 NS experts.  positions[] receives the slot's rank among
// its block's rows of the expert (the final row when there is one block).
template <int NS>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(RouteArgs a) {
    __shared__ int run[kRouteMaxExperts];                       // rows of each expert before the pass
    __shared__ uint32_t mask[kRouteWords][kRouteMaxExperts];    // tokens of the pass that chose it
    __shared__ int16_t picks[kRoutePass][kRouteMaxTopK];
    __shared__ int base[kRouteMaxExperts + 1];
    __shared__ int warp_sums[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) {
        run[e] = 0;
#pragma unroll
        for (int w = 0; w < kRouteWords; ++w) mask[w][e] = 0;
    }
    __syncthreads();
    sm100::grid_dependency_pass();
    const int t_begin = blockIdx.x * a.per_block;
    const int t_end = min(a.T, t_begin + a.per_block);
    for (int t0 = t_begin; t0 < t_end; t0 += kRoutePass) {
#pragma unroll 1
        for (int w = 0; w < kRouteWords; ++w) {
            const int t = t0 + w * 32 + warp;
            if (t >= t_end) break;
            uint32_t key[NS];
            int slot[NS];
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int e = s * 32 + lane;
                key[s] = 0;
                slot[s] = s;
                if (e < a.E)
                    key[s] = logit_key(a.half ? h2f(static_cast<const uint16_t*>(a.logits)[t * a.ld + e])
                                              : static_cast<const float*>(a.logits)[t * a.ld + e]);
            }
            // softmax over every expert that is not masked: exp(l - top), +inf as the largest finite value
            uint32_t head = 0;
#pragma unroll
            for (int s = 0; s < NS; ++s) head = max(head, key[s]);
            uint32_t top = __reduce_max_sync(0xffffffffu, head);
            const float lmax = top ? fminf(key_logit(top), 3.402823466e38f) : 0.0f;
            float total = 0.0f;
            if (!a.sigmoid && !a.renorm) {
#pragma unroll
                for (int s = 0; s < NS; ++s)
                    if (key[s]) total += expf(fminf(key_logit(key[s]), 3.402823466e38f) - lmax);
#pragma unroll
                for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
            }
            int chosen = -1;
            uint32_t chosen_key = 0;
            constexpr bool kSorted = NS <= 4;       // (a longer sort costs more than the rounds' scans)
            if constexpr (kSorted) sort_keys(key, slot);
            for (int j = 0; j < a.k; ++j) {
                int be;
                if constexpr (kSorted) {
                    head = key[0];
                    be = slot[0] * 32 + lane;
                } else {
                    head = 0;
                    be = 0;
#pragma unroll
                    for (int s = 0; s < NS; ++s)
                        if (key[s] > head) head = key[s], be = s * 32 + lane;
                }
                top = __reduce_max_sync(0xffffffffu, head);
                if (top == 0) break;                                  // only masked experts are left
                const int we = (int)__reduce_min_sync(0xffffffffu, head == top ? (uint32_t)be : 0x7fffffffu);
                if (lane == j) chosen = we, chosen_key = top;
                if (head == top && be == we) {                        // the winner's lane drops its head
                    if constexpr (kSorted) {
#pragma unroll
                        for (int s = 0; s + 1 < NS; ++s) key[s] = key[s + 1], slot[s] = slot[s + 1];
                        key[NS - 1] = 0;
                    } else {
#pragma unroll
                        for (int s = 0; s < NS; ++s)
                            if (we == s * 32 + lane) key[s] = 0;
                    }
                }
                __syncwarp();
            }
            float v = 0.0f;
            if (chosen >= 0) {
                const float l = fminf(key_logit(chosen_key), 3.402823466e38f);
                v = a.sigmoid ? sigmoid_score(l, a.renorm ? fminf(lmax, 0.0f) : 0.0f) : expf(l - lmax);
                if (!a.sigmoid && !a.renorm) v /= total;
            }
            if (a.renorm) {
                float sum = v;
#pragma unroll
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                v = sum > 0.0f ? v / sum : 0.0f;
            }
            if (lane < a.k) {
                a.weights[(size_t)t * a.k + lane] = v;
                a.experts[(size_t)t * a.k + lane] = chosen;
                picks[w * 32 + warp][lane] = (int16_t)chosen;
            }
            if (chosen >= 0) atomicOr(&mask[w][chosen], 1u << warp);
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kRouteWords; ++w) {
            const int t = t0 + w * 32 + warp;
            if (t < t_end && lane < a.k) {
                const int e = picks[w * 32 + warp][lane];
                int rank = -1;
                if (e >= 0) {
                    rank = run[e] + __popc(mask[w][e] & ((1u << warp) - 1u));
                    for (int v = 0; v < w; ++v) rank += __popc(mask[v][e]);
                }
                a.positions[(size_t)t * a.k + lane] = rank;
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += kRouteThreads) {
            int n = run[e];
#pragma unroll
            for (int w = 0; w < kRouteWords; ++w) {
                n += __popc(mask[w][e]);
                mask[w][e] = 0;
            }
            run[e] = n;
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

// Four lanes per token, for top_k <= KT (2, 4 or 8): each lane walks a quarter of the row
// and keeps its KT largest in registers, one compare and a shift per slot; two bitonic merges make the
// token's list.  8 tokens share each instruction (about 200 a token at 128 experts and KT = 8, against 610
// for the warp form, whose reductions serve one token); a single lane per token needs no merge, but 16384
// tokens are then less than one warp per scheduler.  Same ranks and counts.
constexpr int kRouteWalkThreads = 4 * kRoutePass;

// (key, expert) as one number that falls in the order of the choice: larger key, then lower expert.
__device__ __forceinline__ unsigned long long route_rank(uint32_t key, int e) {
    return (unsigned long long)key << 32 | (uint32_t)~e;
}

template <int KT>
__global__ void __launch_bounds__(kRouteWalkThreads) route_walk_kernel(RouteArgs a) {
    __shared__ int run[kRouteMaxExperts];
    __shared__ uint32_t mask[kRouteWords][kRouteMaxExperts];
    const int q = threadIdx.x & 3, tok = threadIdx.x >> 2;          // lane of the token, token of the pass
    const int word = tok >> 5;
    const uint32_t bit = 1u << (tok & 31);
    for (int e = threadIdx.x; e < a.E; e += kRouteWalkThreads) {
        run[e] = 0;
#pragma unroll
        for (int w = 0; w < kRouteWords; ++w) mask[w][e] = 0;
    }
    __syncthreads();
    sm100::grid_dependency_pass();
    const int t_begin = blockIdx.x * a.per_block;
    const int t_end = min(a.T, t_begin + a.per_block);
    constexpr int kOwn = (KT + 3) / 4;                              // slots that a lane writes
    for (int t0 = t_begin; t0 < t_end; t0 += kRoutePass) {
        const int t = t0 + tok;
        const bool live = t < t_end;
        uint32_t key[KT] = {};          // falling; equal keys in rising expert order; 0: none
        int pick[KT];
#pragma unroll
        for (int s = 0; s < KT; ++s) pick[s] = -1;
        const char* row = static_cast<const char*>(a.logits) + (size_t)(live ? t : t_begin) * a.ld * (a.half ? 2 : 4);
        auto insert = [&](float l, int e) {
            const uint32_t n = logit_key(l);
            bool above[KT];                             // n goes before slot s
#pragma unroll
            for (int s = 0; s < KT; ++s) above[s] = n > key[s];
#pragma unroll
            for (int s = KT - 1; s > 0; --s) {
                key[s] = above[s - 1] ? key[s - 1] : (above[s] ? n : key[s]);
                pick[s] = above[s - 1] ? pick[s - 1] : (above[s] ? e : pick[s]);
            }
            key[0] = above[0] ? n : key[0];
            pick[0] = above[0] ? e : pick[0];
        };
        // a token's lanes take turns of 16 bytes where the rows allow it, of one expert otherwise
        int e = 0;
        if ((reinterpret_cast<uintptr_t>(row) & 15) == 0) {
            if (a.half) {
                for (; e + 32 <= a.E; e += 32) {
                    const uint4 v = *reinterpret_cast<const uint4*>(row + (e + q * 8) * 2);
                    const uint16_t* h = reinterpret_cast<const uint16_t*>(&v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) insert(h2f(h[i]), e + q * 8 + i);
                }
            } else {
                for (; e + 16 <= a.E; e += 16) {
                    const float4 v = *reinterpret_cast<const float4*>(row + (e + q * 4) * 4);
                    const int e0 = e + q * 4;
                    insert(v.x, e0), insert(v.y, e0 + 1), insert(v.z, e0 + 2), insert(v.w, e0 + 3);
                }
            }
        }
#pragma unroll 1
        for (e += q; e < a.E; e += 4)
            insert(a.half ? h2f(reinterpret_cast<const uint16_t*>(row)[e]) : reinterpret_cast<const float*>(row)[e], e);
        __syncwarp();
        // merge with the neighbour's list, then with the other pair's: the larger of (mine i, theirs KT-1-i)
        // are the KT largest of both, in bitonic order
#pragma unroll
        for (int x = 1; x <= 2; x <<= 1) {
            unsigned long long v[KT];
#pragma unroll
            for (int s = 0; s < KT; ++s) v[s] = route_rank(key[s], pick[s]);
            unsigned long long o[KT];
#pragma unroll
            for (int s = 0; s < KT; ++s) o[s] = __shfl_xor_sync(0xffffffffu, v[KT - 1 - s], x);
#pragma unroll
            for (int s = 0; s < KT; ++s) v[s] = max(v[s], o[s]);
#pragma unroll
            for (int d = KT / 2; d; d >>= 1)
#pragma unroll
                for (int s = 0; s < KT; ++s)
                    if (!(s & d)) {
                        const unsigned long long hi = max(v[s], v[s + d]), lo = min(v[s], v[s + d]);
                        v[s] = hi, v[s + d] = lo;
                    }
#pragma unroll
            for (int s = 0; s < KT; ++s) key[s] = (uint32_t)(v[s] >> 32), pick[s] = key[s] ? (int)~(uint32_t)v[s] : -1;
        }
        const float lmax = key[0] ? fminf(key_logit(key[0]), 3.402823466e38f) : 0.0f;
        float total = 0.0f;
        if (!a.sigmoid && !a.renorm) {
#pragma unroll 4
            for (e = q; e < a.E; e += 4) {
                const float l = a.half ? h2f(reinterpret_cast<const uint16_t*>(row)[e]) : reinterpret_cast<const float*>(row)[e];
                if (logit_key(l)) total += expf(fminf(l, 3.402823466e38f) - lmax);
            }
            __syncwarp();
            total += __shfl_xor_sync(0xffffffffu, total, 1);
            total += __shfl_xor_sync(0xffffffffu, total, 2);
        }
        // lane q writes slots q kOwn .. q kOwn + kOwn - 1
        float w[kOwn], sum = 0.0f;
        int own[kOwn];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            uint32_t k = 0;
            own[i] = -1;
            w[i] = 0.0f;
#pragma unroll
            for (int s = 0; s < KT; ++s)
                if (s == q * kOwn + i && s < a.k) k = key[s], own[i] = pick[s];
            if (k) {
                const float l = fminf(key_logit(k), 3.402823466e38f);
                w[i] = a.sigmoid ? sigmoid_score(l, a.renorm ? fminf(lmax, 0.0f) : 0.0f) : expf(l - lmax);
                if (!a.sigmoid && !a.renorm) w[i] /= total;
            }
            sum += w[i];
        }
        __syncwarp();
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int s = q * kOwn + i;
            if (live && s < a.k) {
                if (a.renorm) w[i] = sum > 0.0f ? w[i] / sum : 0.0f;
                a.weights[(size_t)t * a.k + s] = w[i];
                a.experts[(size_t)t * a.k + s] = own[i];
                if (own[i] >= 0) atomicOr(&mask[word][own[i]], bit);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int s = q * kOwn + i;
            if (live && s < a.k) {
                int rank = -1;
                if (own[i] >= 0) {
                    rank = run[own[i]] + __popc(mask[word][own[i]] & (bit - 1u));
                    for (int v = 0; v < word; ++v) rank += __popc(mask[v][own[i]]);
                }
                a.positions[(size_t)t * a.k + s] = rank;
            }
        }
        __syncthreads();
        for (e = threadIdx.x; e < a.E; e += kRouteWalkThreads) {
            int n = run[e];
#pragma unroll
            for (int v = 0; v < kRouteWords; ++v) {
                n += __popc(mask[v][e]);
                mask[v][e] = 0;
            }
            run[e] = n;
        }
        __syncthreads();
    }
    for (int e = threadIdx.x; e < a.E; e += kRouteWalkThreads)
        a.counts[(size_t)blockIdx.x * a.E + e] = (uint16_t)run[e];
}

// Second step: every block adds the counts of the blocks before it and turns its slots' ranks
// into rows.
__global__ void __launch_bounds__(kRouteThreads) route_order_kernel(RouteArgs a) {
    __shared__ int total[kRouteMaxExperts], before[kRouteMaxExperts];
    __shared__ int base[kRouteMaxExperts + 1];
    __shared__ int warp_sums[32];
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) total[e] = before[e] = 0;
    __syncthreads();
    sm100::grid_dependency_pass();
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
        per_block = ceil_div(T, 32) * 32;
        return 1;
    }
    per_block = std::min(ceil_div(ceil_div(T, sms), 32) * 32, 65504);     // (counts are 16 bits)
    return ceil_div(T, per_block);
}

inline size_t route_workspace_bytes(int T, int E, int sms) {
    if (T <= 0 || E <= 0) return 0;
    int per = 0;
    const int blocks = route_blocks(T, sms, per);
    return blocks > 1 ? align256((size_t)blocks * E * 2) : 0;
}

// Whether four lanes take a token instead of a warp (several blocks, top_k <= 8).  Measured, warp / four lanes, us:
//   top 2 of 8:   256 tokens 5.9 / 5.2, 4096 6.3 / 5.4, 16384 11.1 / 5.6;    top 4 of 32: 256 5.9 / 5.9, 16384 12.9 / 7.3
//   top 4 of 64:  256 6.3 / 6.8, 4096 7.7 / 7.8, 8192 9.8 / 8.0;  top 2 of 128: 256 7.0 / 7.0, 4096 8.3 / 8.2, 8192 11.0 / 8.4
//   top 8 of 128: 256 7.7 / 12.6, 8192 12.7 / 14.4, 10240 16.8 / 15.4, 16384 19.4 / 14.9
inline bool route_by_walk(const RouteArgs& a) {
    if (a.blocks == 1 || a.k > 8) return false;
    return a.E * a.k <= 128 || a.T >= (a.k <= 4 ? 6144 : 9216);
}

inline awq_status launch_route(RouteArgs a, cudaStream_t st) {
    const void* fn = a.E <= 32    ? (const void*)route_kernel<1>
                     : a.E <= 64  ? (const void*)route_kernel<2>
                     : a.E <= 128 ? (const void*)route_kernel<4>
                     : a.E <= 256 ? (const void*)route_kernel<8>
                     : a.E <= 512 ? (const void*)route_kernel<16>
                                  : (const void*)route_kernel<32>;
    void* args[] = {&a};
    int threads = kRouteThreads;
    if (route_by_walk(a)) {
        fn = a.k <= 2   ? (const void*)route_walk_kernel<2>
             : a.k <= 4 ? (const void*)route_walk_kernel<4>
                        : (const void*)route_walk_kernel<8>;
        threads = kRouteWalkThreads;
    }
    if (!launch_pdl(fn, dim3((unsigned)a.blocks), dim3(threads), args, st)) return AWQ_ERR_CUDA;
    if (a.blocks > 1 &&
        !launch_pdl((const void*)route_order_kernel, dim3((unsigned)a.blocks), dim3(kRouteThreads), args, st))
        return AWQ_ERR_CUDA;
    return AWQ_OK;
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
    sm100::grid_dependency_pass();
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
    const int V = (a & 15) == 0 ? 8 : ((a & 3) == 0 ? 2 : 1);
    const void* fn = V == 8   ? (const void*)combine_kernel<8>
                     : V == 2 ? (const void*)combine_kernel<2>
                              : (const void*)combine_kernel<1>;
    const dim3 grid((unsigned)T, ceil_div(N, kCombineThreads * V));
    void* args[] = {&Y, &R, &ldy, &weights, &positions, &k, &N, &residual, &ldr, &out, &ldo};
    return launch_pdl(fn, grid, dim3(kCombineThreads), args, st) ? AWQ_OK : AWQ_ERR_CUDA;
}

}  // namespace awq
