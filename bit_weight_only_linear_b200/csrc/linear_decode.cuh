// Fused linear and expert-grouped linear for few rows (decode): HBM-bound streaming of the packed
// weights past the rows of X, multiplied with mma.sync straight from registers.
//
// The arithmetic is the GEMV's (gemv.cuh): a mask turns two adjacent codes into fp16 subnormals
// q 2^-24 (or 16 q 2^-24), m16n8k16 multiplies them exactly with up to 8 rows of X, and the group's
// scale and zero point are applied once per k-step in fp32, so no weight is rounded:
//     y += (scale16 2^24) (D1 + D16 / 16) - (scale16 z) sum_k x.
// What differs is the shape of the work:
//   * A unit is 32 weight rows (two MMA row tiles) by the whole K.  The two tiles share every X
//     fragment, which halves the shared-memory reads of X per weight (they, not the weights, bound
//     the 16-row form at 8 rows).  Gated, the tiles are 16 gate rows and the 16 rows F behind them,
//     so both halves of an output meet in one unit's partial sums.
//   * A persistent CTA per SM takes a contiguous range of units: all of one dense matrix, or the
//     units of the experts that have rows (8 rows of an expert at a time), so that X is staged once
//     per expert and CTA.
//   * With many units per CTA a unit is 64 rows and a stage 64 rows x 1024 codes (RS = 2): 8 warps split
//     the K of each half, so half as many partial sums meet per row.  With few, 32 rows (RS = 1) share out
//     more evenly.
//   * Warps: a producer (3-D TMA, 32 KB stages of 32 rows x 2048 codes), two converters (scales and
//     zeros -> fp32 pairs per stage), 16 consumers (128 codes of a stage each), a reducer for each 32
//     rows of the unit (the consumers' partial sums in a fixed order, then the epilogue).
// Bound: HBM where CTAs get many units (8 tokens, 2 of 8 experts, 28672 x 4096: 367 MB of the 6 experts touched
// in 69.7 us = 5.26 TB/s, 0.80 of the measured copy rate); for one dense matrix the start and end of a launch,
// about 4 us, and the uneven last unit (1 row x 28672 x 4096, gated: 15.2 us = 4.0 TB/s; 4096 x 4096: 4.7 us).
// The GEMV, without an epilogue, is 4 to 8 % faster at one row (13.4 against 14.5 us for 28672 x 4096, 4.35
// against 4.7 for 4096 x 4096: two CTAs an SM and 16-row units) and slower from 2 to 4 rows on (8 rows: 19.9
// against 16.9, 8.0 against 6.8).
// K must be a multiple of 128.  Every wait is bounded.
#pragma once

#include "common.cuh"
#include "epilogue.cuh"
#include "gemv.cuh"
#include "gemv_launch.cuh"
#include "linear_common.cuh"
#include "linear_tc.cuh"
#include "sm100.cuh"

namespace awq {

constexpr int kDecConsumers = 16;
constexpr int kDecConverters = 2;
constexpr int kDecReducer0 = 1 + kDecConverters;  // first reducer's warp; RS reducers, then the consumers
constexpr int dec_threads(int RS) { return (kDecReducer0 + RS + kDecConsumers) * 32; }
constexpr int kDecRows = 32;                     // weight rows of a consumer: two MMA row tiles
constexpr int kDecStageBytes = 32 * 1024;        // 32 RS rows x 2048 / RS codes
constexpr int kDecMaxRows = 8;                   // rows of X at a time (MMA N)
constexpr int kDecManyUnits = 8;                 // 32-row units (gated: pairs of them) per CTA from which a unit is 64 rows
constexpr int kDecMaxSegs = 32;                  // segments of a CTA
constexpr int kDecMaxK = 1 << 17;                // (no row of X beyond it fits in shared memory)
constexpr int kDecPartPitch = 36;                // words per row of X in a partial sum (bank spread)

struct DecSmem {
    int K, M, S, RS, Kp, nsteps, gpc;
    __host__ __device__ DecSmem(int M_, int K_, int G, int S_, int RS_) : K(K_), M(M_), S(S_), RS(RS_) {
        const int kc = 2048 / RS;                // codes per row and stage
        Kp = (K + kc - 1) / kc * kc;
        nsteps = Kp / (32 * gemv_words_per_thread(G));
        gpc = kc / G;
    }
    // converted (scale, scale * zero) pairs of a stage: [32 RS rows][gpc], rows padded by 16 bytes
    __host__ __device__ int cvt_pitch() const { return gpc * 8 + 16; }
    __host__ __device__ int cvt() const { return S * kDecStageBytes; }
    __host__ __device__ int x() const { return cvt() + S * kDecRows * RS * cvt_pitch(); }
    __host__ __device__ int x_pitch() const { return Kp * 2 + 64; }
    __host__ __device__ int xsum() const { return x() + M * x_pitch(); }
    __host__ __device__ int part() const { return (xsum() + M * nsteps * 4 + 15) & ~15; }
    __host__ __device__ int part_stride() const { return kDecConsumers * M * kDecPartPitch * 4; }
    __host__ __device__ int bars() const { return part() + 2 * part_stride(); }
    // full[S], empty[S], rfull[2], rempty[2], abort flag and segment count, segments
    __host__ __device__ int segs() const { return bars() + (2 * S + 4) * 8 + 8; }
    __host__ __device__ int bytes() const { return segs() + kDecMaxSegs * 20; }
};

struct DecArgs {
    const uint16_t* X;
    long long ldx;
    const uint16_t* scales;
    const uint32_t* qzeros;              // NULL: implicit zero 8
    const int32_t* rows;                 // row numbers of X, or NULL
    const int32_t* offsets;              // [E+1], or NULL: one range of R rows
    int T, R, E, N, K;
    int units;                           // units of one matrix
    int mc;                              // rows of X at a time
    int S;                               // stages
    Epilogue ep;
};

// A run of units of one matrix with one set of rows.
struct DecSeg {
    int expert, r0, nr, n, count;        // rows r0 .. r0+nr-1; units n .. n+count-1
};

// Row sets (of up to mc rows) of all experts, by a whole warp.
__device__ __forceinline__ int dec_sets(const DecArgs& a) {
    if (!a.offsets) return ceil_div(a.R, a.mc);
    int t = 0;
    for (int e = threadIdx.x & 31; e < a.E; e += 32) {
        const int2 g = expert_range(a.offsets, e, a.R);
        t += (g.y - g.x + a.mc - 1) / a.mc;
    }
    return __reduce_add_sync(0xffffffffu, t);
}

// The segment that starts at unit u (of all sets' units, set by set), at most up to unit `end`.
__device__ __forceinline__ DecSeg dec_segment(const DecArgs& a, int u, int end) {
    const int set = u / a.units;
    DecSeg s;
    s.n = u - set * a.units;
    s.count = min(a.units - s.n, end - u);
    if (a.offsets) {
        const int4 t = find_tile(a.offsets, a.E, a.R, a.mc, 1, 1, set);
        s.expert = t.x;
        s.r0 = t.y;
        s.nr = t.z - t.y;
    } else {
        s.expert = 0;
        s.r0 = set * a.mc;
        s.nr = min(a.mc, a.R - s.r0);
    }
    return s;
}

// The stages of a CTA's segments in order.
struct DecIter {
    const DecSeg *sg, *end;
    int n, c, nchunks;
    __device__ __forceinline__ DecIter(const DecSeg* segs, int count, int nchunks_)
        : sg(segs), end(segs + count), n(0), c(0), nchunks(nchunks_) {
        if (live()) n = sg->n;
    }
    __device__ __forceinline__ bool live() const { return sg < end; }
    __device__ __forceinline__ void next() {
        if (!live() || ++c < nchunks) return;
        c = 0;
        if (++n < sg->n + sg->count) return;
        if (++sg < end) n = sg->n;
    }
};

template <int G, int RS>
__global__ void __launch_bounds__(dec_threads(RS), 1)
linear_decode_kernel(const __grid_constant__ CUtensorMap tmap_q, const DecArgs a) {
    using namespace sm100;
    constexpr int WT = gemv_words_per_thread(G);
    constexpr int kStepCodes = 32 * WT;
    constexpr int Q = 128 / kStepCodes;                    // k-steps of a consumer per stage
    constexpr int KC = 2048 / RS;                          // codes per row and stage
    constexpr int GPC = KC / G;                            // groups per row and stage
    constexpr int KS = kDecConsumers / RS;                 // consumers that share the K of 32 rows
    constexpr int kConsumer0 = kDecReducer0 + RS;          // first consumer's warp
    constexpr int kSub = kDecStageBytes / RS;              // their part of a stage
    extern __shared__ __align__(128) uint8_t smem[];
    const DecSmem L(a.mc, a.K, G, a.S, RS);
    const int S = a.S;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L.bars());   // weights and converted pairs in
    uint64_t* empty = full + S;                    // consumers done with a stage
    uint64_t* rfull = empty + S;                   // partial sums of a unit written
    uint64_t* rempty = rfull + 2;                  // reducer done with the slot
    volatile uint32_t* abort = reinterpret_cast<volatile uint32_t*>(rempty + 2);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 2);                // producer (with its bytes) + converter
            mbar_init(&empty[i], kDecConsumers);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&rfull[i], kDecConsumers);
            mbar_init(&rempty[i], RS);
        }
        *abort = 0;
        mbar_fence_init();
        prefetch_tensormap(&tmap_q);
    }
    // Grouped, the table decides which weights are read; dense, the weights stream before the previous
    // kernel has completed, and only X, the residual and Y wait for it (below).
    if (a.offsets) grid_dependency_pass();
    DecSeg* segs = reinterpret_cast<DecSeg*>(smem + L.segs());
    if (warp == 1) {
        // this CTA's share of all row sets' units, as segments
        const long long total = min((long long)dec_sets(a) * a.units, 0x7fffffffLL);
        const int u_begin = (int)(total * blockIdx.x / gridDim.x), u_end = (int)(total * (blockIdx.x + 1) / gridDim.x);
        int count = 0;
        for (int u = u_begin; u < u_end && count < kDecMaxSegs; ++count) {
            const DecSeg sg = dec_segment(a, u, u_end);
            if (lane == 0) segs[count] = sg;
            u += sg.count;
        }
        if (lane == 0) abort[1] = (uint32_t)count;
    }
    __syncthreads();
    const int nseg = (int)abort[1];
    const int nchunks = L.Kp / KC;
    const int F = a.ep.gated ? a.N / 2 : a.N;
    const uint32_t sbase = smem_u32(smem);
    // first rows of the two row tiles of part p of unit n
    auto tile0 = [&](int n, int p) { return (n * RS + p) * (a.ep.gated ? 16 : 32); };
    auto tile1 = [&](int n, int p) { return a.ep.gated ? F + (n * RS + p) * 16 : (n * RS + p) * 32 + 16; };

    if (warp == 0) {
        // ---------------- producer ----------------
        int st = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int i = 0; i < nseg && ok; ++i) {
            const DecSeg sg = segs[i];
            for (int n = sg.n; n < sg.n + sg.count && ok; ++n) {
                for (int c = 0; c < nchunks; ++c) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], ph ^ 1u));
                    if (!ok) break;
                    if (elect_one()) {
                        uint8_t* dst = smem + (size_t)st * kDecStageBytes;
                        // boxes {16 words, 16 rows, KC / 128 blocks of 128 codes}; blocks past K are zeros
                        mbar_arrive_expect_tx(&full[st], kDecStageBytes);
#pragma unroll
                        for (int p = 0; p < RS; ++p) {
                            tma_load_3d(dst + p * kSub, &tmap_q, &full[st], 0, sg.expert * a.N + tile0(n, p), c * (KC / 128));
                            tma_load_3d(dst + p * kSub + kSub / 2, &tmap_q, &full[st], 0, sg.expert * a.N + tile1(n, p),
                                        c * (KC / 128));
                        }
                    }
                    __syncwarp();
                    ++issued;
                    if (++st == S) st = 0, ph ^= 1u;
                }
            }
        }
        // copies in flight must land before the CTA exits
        for (int j = issued - 1; j >= 0 && j >= issued - S; --j) mbar_wait(&full[j % S], (j / S) & 1);
        return;
    }
    if (warp < kDecReducer0) {
        // ---------------- converters: lane = row of each part of the unit.  Each takes every second stage and holds
        // the scales and zero words of the next kDepth of them in registers (a stage's loads take longer
        // than the stage streams) ----------------
        static_assert(GPC % 8 == 0, "whole octets of groups per row and stage");
        constexpr int OPR = GPC / 8, OCT = RS * OPR;           // octets of groups per row, per lane and stage
        constexpr int kDepth = OCT <= 4 ? 2 : 1;
        const int ng = a.K / G, nzw = ceil_div(ng, 8);
        const bool zp = a.qzeros != nullptr;
        const bool vec = (ng & 7) == 0;                        // 16-byte aligned scale rows
        uint4 sc[kDepth][OCT];
        uint32_t zw[kDepth][OCT];
        auto fetch = [&](const DecIter& it, uint4 (&fs)[OCT], uint32_t (&fz)[OCT]) {
            if (!it.live()) return;
#pragma unroll
            for (int o = 0; o < OCT; ++o) {
                const int p = o / OPR;
                const int row = lane < 16 ? tile0(it.n, p) + lane : tile1(it.n, p) + lane - 16;
                const int lim = a.ep.gated && lane < 16 ? F : a.N;
                const size_t wr = (size_t)it.sg->expert * a.N + min(row, lim - 1);   // rows past the end: dropped later
                const uint16_t* sp = a.scales + wr * ng;
                const int g0 = it.c * GPC + 8 * (o % OPR);
                fs[o] = make_uint4(0u, 0u, 0u, 0u);                                  // groups past K: scale 0
                fz[o] = 0x88888888u;
                if (g0 < ng) {
                    if (vec) {
                        fs[o] = __ldg(reinterpret_cast<const uint4*>(sp + g0));
                    } else if ((ng & 1) == 0) {
                        // rows of other lengths in words or halves, all loads in flight together (one after the
                        // other they took longer than the stage: 34 experts x 2048 x 1408, G = 64: 39 us)
                        const uint32_t* wp = reinterpret_cast<const uint32_t*>(sp + g0);
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = g0 + 2 * i < ng ? __ldg(wp + i) : 0u;
                        fs[o] = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
                        uint32_t h[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) h[i] = g0 + i < ng ? __ldg(sp + g0 + i) : 0u;
                        fs[o] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
                    }
                    if (zp) fz[o] = __ldg(a.qzeros + wr * nzw + (g0 >> 3));
                }
            }
        };
        DecIter fetched(segs, nseg, nchunks);                 // the next stage to fetch
        DecIter it(segs, nseg, nchunks);                      // the next to convert
        if (warp == 2) fetched.next(), it.next();
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            fetch(fetched, sc[d], zw[d]);
            fetched.next();
            fetched.next();
        }
        int st = warp - 1;
        uint32_t ph = 0;
        while (it.live()) {
#pragma unroll
            for (int d = 0; d < kDepth; ++d) {
                if (!it.live()) break;
                mbar_wait_or_abort(&empty[st], ph ^ 1u, abort);
                uint8_t* rows = smem + L.cvt() + (st * RS * kDecRows + lane) * L.cvt_pitch();
#pragma unroll
                for (int o = 0; o < OCT; ++o) {
                    float4* dst = reinterpret_cast<float4*>(rows + o / OPR * kDecRows * L.cvt_pitch()) + o % OPR * 4;
                    const uint32_t hw[4] = {sc[d][o].x, sc[d][o].y, sc[d][o].z, sc[d][o].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float s0 = h2f((uint16_t)(hw[k] & 0xFFFFu)), s1 = h2f((uint16_t)(hw[k] >> 16));
                        const float z0 = (float)((zw[d][o] >> (8 * k)) & 15u), z1 = (float)((zw[d][o] >> (8 * k + 4)) & 15u);
                        dst[k] = make_float4(s0 * 16777216.0f, s0 * z0, s1 * 16777216.0f, s1 * z1);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[st]);
                st += kDecConverters;
                if (st >= S) st -= S, ph ^= 1u;
                it.next();
                it.next();
                fetch(fetched, sc[d], zw[d]);
                fetched.next();
                fetched.next();
            }
        }
        return;
    }
    if (warp < kConsumer0) {
        // ---------------- reducers: the consumers' sums in order, then the epilogue.  Lane = (row of X,
        // four weight rows); 16-byte reads, all independent.  A warp for each 32 rows of the unit: with one for
        // both, the chain of reads, activation and stores took longer than the weights where K is short
        // (3 rows each of 64 experts, 2816 x 2048, gated: 51 -> 40 us; with three or more the consumers have too
        // few registers: 43) ----------------
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const Epilogue& ep = a.ep;
        const int quad = lane & 7;
        int b = 0;
        uint32_t ph = 0;
        for (int i = 0; i < nseg; ++i) {
            const DecSeg sg = segs[i];
            const uint16_t* bias = ep.bias ? ep.bias + (size_t)sg.expert * a.N : nullptr;
            for (int n = sg.n; n < sg.n + sg.count; ++n) {
                mbar_wait_or_abort(&rfull[b], ph, abort);
                __syncwarp();
                const uint32_t slot = sbase + (uint32_t)(L.part() + b * L.part_stride() + quad * 16);
                const int p = warp - kDecReducer0;
                const int row = quad < 4 ? tile0(n, p) + quad * 4 : tile1(n, p) + quad * 4 - 16;
                const int lim = ep.gated && quad < 4 ? F : a.N;
                float bv[4] = {};
                if (bias) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (row + i < lim) bv[i] = h2f(__ldg(bias + row + i));
                }
                // (not unrolled, here and in the other rare paths: the roles share the instruction cache, and
                // what they fetch anew for every unit shows: 61 -> 55 us on 64 experts of 3 rows; 8-byte stores
                // with a second path for odd strides gain nothing)
#pragma unroll 1
                for (int it = 0; it * 4 < sg.nr; ++it) {
                    const int m = it * 4 + (lane >> 3), mm = min(m, sg.nr - 1);
                    const bool store = m < sg.nr && (!ep.gated || quad < 4);
                    float y[4] = {}, res[4] = {}, other[4];
                    if (ep.residual && store) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (row + i < lim) res[i] = h2f(ep.residual[(size_t)(sg.r0 + m) * ep.ldr + row + i]);
                    }
#pragma unroll
                    for (int w = 0; w < KS; ++w) {
                        const uint4 v = lds128(slot + (uint32_t)(((p * KS + w) * a.mc + mm) * kDecPartPitch * 4));
                        y[0] += __uint_as_float(v.x), y[1] += __uint_as_float(v.y);
                        y[2] += __uint_as_float(v.z), y[3] += __uint_as_float(v.w);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[i] += bv[i];
                        other[i] = __shfl_down_sync(0xffffffffu, y[i], 4);
                    }
                    apply_act(y, ep.act);
                    uint16_t* yp = ep.Y + (size_t)(sg.r0 + m) * ep.ldy + row;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (ep.gated) y[i] *= other[i];
                        if (store && row + i < lim) yp[i] = f2h_rn(y[i] + res[i]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&rempty[b]);
                if (++b == 2) b = 0, ph ^= 1u;
            }
        }
        return;
    }

    // ---------------- consumers ----------------
    constexpr int kCons = kDecConsumers * 32;
    constexpr int R = G >= kStepCodes ? G / kStepCodes : 1;     // k-steps per group
    constexpr int TPS = 4 * WT;                                  // 16-byte chunks per k-step
    const int cw = warp - kConsumer0, ct = threadIdx.x - kConsumer0 * 32;
    const int g = lane >> 2, t = lane & 3;
    const int pitch = L.x_pitch();
    uint8_t* xs = smem + L.x();
    float* xsum = reinterpret_cast<float*>(smem + L.xsum());
    const int part = cw / KS, ks = cw % KS;         // part of the unit, block of 128 codes of a stage
    // weights: row r of a tile, block b of 128 codes: [b][r][64 bytes]
    const uint32_t wofs = (uint32_t)(part * kSub + ks * 1024 + g * 64 + t * WT * 4);
    const uint32_t cofs =
        smem_u32(smem + L.cvt()) + (uint32_t)((part * kDecRows + g) * L.cvt_pitch() + (ks * 128 / G) * 8);
    const uint32_t crow8 = 8u * L.cvt_pitch(), cstage = (uint32_t)(RS * kDecRows * L.cvt_pitch());
    const int m0 = 2 * t, m1 = 2 * t + 1;
    int st = 0, b = 0;
    uint32_t ph = 0, rph = 0;
    grid_dependency_pass();
    for (int i = 0; i < nseg; ++i) {
        const DecSeg sg = segs[i];
        // X of the segment: 16-byte chunks reordered within each k-step to [j][t] with the middle words
        // swapped (so that a fragment is a register pair of one 16-byte read), zeros past K and for rows
        // that do not exist; per-k-step sums of x
        asm volatile("bar.sync 1, %0;" ::"n"(kCons) : "memory");       // the previous segment's X is done with
        {
            const int kwp = L.Kp >> 3, kwv = a.K >> 3;                 // kwp is a multiple of 128
            constexpr int kBatch = 4;                                  // rows whose loads are in flight together
#pragma unroll 1
            for (int mb = 0; mb < sg.nr; mb += kBatch) {
                const uint4* row[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    int src = -1;
                    if (mb + i < sg.nr) src = a.rows ? __ldg(a.rows + sg.r0 + mb + i) : sg.r0 + mb + i;
                    row[i] = src >= 0 && src < a.T ? reinterpret_cast<const uint4*>(a.X + src * a.ldx) : nullptr;
                }
#pragma unroll 1
                for (int word = ct; word < kwp; word += kCons) {
                    const int s = word / TPS, r = word % TPS;
                    const int tt = r / WT, j = r % WT;
                    uint4 v[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        v[i] = row[i] && word < kwv ? __ldg(row[i] + word) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const int m = mb + i;
                        if (m >= sg.nr) break;
                        reinterpret_cast<uint4*>(xs + m * pitch)[(s * WT + j) * 4 + tt] =
                            make_uint4(v[i].x, v[i].z, v[i].y, v[i].w);
                        const uint16_t* h = reinterpret_cast<const uint16_t*>(&v[i]);
                        float acc = 0.0f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) acc += h2f(h[e]);
#pragma unroll
                        for (int o = TPS / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
                        if (r == 0) xsum[m * L.nsteps + s] = acc;
                    }
                }
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kCons) : "memory");
        // lanes whose column is no row of X read row 0; their sums are not stored
        const uint32_t xrow = smem_u32(xs + (g < sg.nr ? g : 0) * pitch) + (uint32_t)(t * 16 + ks * Q * WT * 64);
        const uint32_t xs0 = smem_u32(xsum + (m0 < sg.nr ? m0 : 0) * L.nsteps + ks * Q);
        const uint32_t xs1 = smem_u32(xsum + (m1 < sg.nr ? m1 : 0) * L.nsteps + ks * Q);
        for (int n = 0; n < sg.count; ++n) {
            float y[2][4] = {};
            for (int c = 0; c < nchunks; ++c) {
                mbar_wait_or_abort(&full[st], ph, abort);
                __syncwarp();
                const uint32_t wb = sbase + (uint32_t)(st * kDecStageBytes) + wofs;
                const uint32_t cv = cofs + (uint32_t)st * cstage;
                const uint32_t xb = xrow + (uint32_t)(c * (KC / kStepCodes) * WT * 64);
                const uint32_t x0b = xs0 + (uint32_t)(c * (KC / kStepCodes) * 4);
                const uint32_t x1b = xs1 + (uint32_t)(c * (KC / kStepCodes) * 4);
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    uint32_t wa[2][WT], wc[2][WT];
                    float d1[2][4], d16[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        lds_words<WT>(wb + h * (kSub / 2) + q * WT * 16, wa[h]);
                        lds_words<WT>(wb + h * (kSub / 2) + 512 + q * WT * 16, wc[h]);
                    }
#pragma unroll
                    for (int j = 0; j < WT; ++j) {
                        const uint4 x = lds128(xb + (uint32_t)((q * WT + j) * 64));
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t p = wa[h][j], r = wc[h][j], p8 = p >> 8, r8 = r >> 8;
                            if (j == 0) {
                                mma_16816_first(d1[h], p & 0x000F000Fu, r & 0x000F000Fu, p8 & 0x000F000Fu,
                                                r8 & 0x000F000Fu, x.x, x.y);
                                mma_16816_first(d16[h], p & 0x00F000F0u, r & 0x00F000F0u, p8 & 0x00F000F0u,
                                                r8 & 0x00F000F0u, x.z, x.w);
                            } else {
                                mma_16816(d1[h], p & 0x000F000Fu, r & 0x000F000Fu, p8 & 0x000F000Fu,
                                          r8 & 0x000F000Fu, x.x, x.y);
                                mma_16816(d16[h], p & 0x00F000F0u, r & 0x00F000F0u, p8 & 0x00F000F0u,
                                          r8 & 0x00F000F0u, x.z, x.w);
                            }
                        }
                    }
                    const float x0 = ldsf(x0b + (uint32_t)(q * 4)), x1 = ldsf(x1b + (uint32_t)(q * 4));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // y += (scale 2^24)(D1 + D16 / 16) - (scale z) sum x
                        const uint32_t at = cv + (uint32_t)((q / R) * 8) + 2u * h * crow8;
                        const uint2 pa = lds64(at), pb = lds64(at + crow8);
                        const float sa = __uint_as_float(pa.x), za = __uint_as_float(pa.y);
                        const float sb = __uint_as_float(pb.x), zb = __uint_as_float(pb.y);
                        y[h][0] = fmaf(sa, fmaf(d16[h][0], 0.0625f, d1[h][0]), fmaf(-za, x0, y[h][0]));
                        y[h][1] = fmaf(sa, fmaf(d16[h][1], 0.0625f, d1[h][1]), fmaf(-za, x1, y[h][1]));
                        y[h][2] = fmaf(sb, fmaf(d16[h][2], 0.0625f, d1[h][2]), fmaf(-zb, x0, y[h][2]));
                        y[h][3] = fmaf(sb, fmaf(d16[h][3], 0.0625f, d1[h][3]), fmaf(-zb, x1, y[h][3]));
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
                if (++st == S) st = 0, ph ^= 1u;
            }
            // the partial sums of the unit: [consumer][row of X][weight row]
            mbar_wait_or_abort(&rempty[b], rph ^ 1u, abort);
            float* pw = reinterpret_cast<float*>(smem + L.part() + b * L.part_stride()) + cw * a.mc * kDecPartPitch + g;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (m0 < sg.nr) {
                    pw[m0 * kDecPartPitch + h * 16] = y[h][0];
                    pw[m0 * kDecPartPitch + h * 16 + 8] = y[h][2];
                }
                if (m1 < sg.nr) {
                    pw[m1 * kDecPartPitch + h * 16] = y[h][1];
                    pw[m1 * kDecPartPitch + h * 16 + 8] = y[h][3];
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&rfull[b]);
            if (++b == 2) b = 0, rph ^= 1u;
        }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Rows of X at a time and stages that fit in `smem` bytes: as many rows as there are, up to 8, with
// at least two stages.  false if not even one row fits.
inline bool dec_plan(int rows, int K, int G, int RS, int smem, int& mc, int& S) {
    for (mc = std::min(rows, kDecMaxRows); mc >= 1; --mc)
        for (S = 6; S >= 2; --S)
            if (DecSmem(mc, K, G, S, RS).bytes() <= smem) return true;
    return false;
}

inline awq_status launch_linear_decode(const LinearArgs& l, const DeviceInfo& d, int RS, int mc, int S,
                                       cudaStream_t st) {
    CUtensorMap tq;
    if (!make_tmap_3d(&tq, l.qweight, CU_TENSOR_MAP_DATA_TYPE_UINT32, 16, (uint64_t)l.E * l.N, (uint64_t)(l.K / 128),
                      (uint64_t)l.K / 2, 64, 16, 16, 2048 / RS / 128))
        return AWQ_ERR_CUDA;
    const void* fn = l.G == 32    ? (RS == 2 ? (const void*)linear_decode_kernel<32, 2> : (const void*)linear_decode_kernel<32, 1>)
                     : l.G == 64  ? (RS == 2 ? (const void*)linear_decode_kernel<64, 2> : (const void*)linear_decode_kernel<64, 1>)
                     : l.G == 128 ? (RS == 2 ? (const void*)linear_decode_kernel<128, 2> : (const void*)linear_decode_kernel<128, 1>)
                                  : (const void*)linear_decode_kernel<256, 1>;
    if (!prepare_kernel(fn)) return AWQ_ERR_CUDA;
    DecArgs a = {l.X, l.ldx, l.scales, l.qzeros, l.rows, l.offsets, l.T, l.R, l.E, l.N, l.K, 0, mc, S, l.ep};
    a.units = l.ep.gated ? ceil_div(l.N / 2, 16 * RS) : ceil_div(l.N, 32 * RS);
    // (grouped: every expert with rows adds at most one partial set)
    const long long sets = l.offsets ? (long long)l.R / mc + std::min(l.R, l.E) : ceil_div(l.R, mc);
    const long long grid = std::min<long long>(d.sms, sets * a.units);
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)grid);
    lc.blockDim = dim3((unsigned)dec_threads(RS));
    lc.dynamicSmemBytes = DecSmem(mc, l.K, l.G, S, RS).bytes();
    lc.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    void* args[] = {&tq, &a};
    return cudaLaunchKernelExC(&lc, fn, args) == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

// Whether 16-row tensor-core tiles, two CTAs to an SM, are the faster form for experts whose units are 64 rows.
// Modelled times (us): a decode stage of 64 rows x 1024 codes takes 0.87 with G = 128 (1.17 where rows of an odd
// number of scales are read by halves), 1.13 with 64 and 1.75 with 32, a unit at least 1.2, and 8 are spent around
// them; a tile's 64 codes take 0.66 to 0.78 while two tiles share an SM, and 9 around them.  Measured, decode against
// tiles, 64 experts of 2048 channels: 3 rows each, G = 128, K = 512 23 / 19, 2048 32 / 44, 4096 53 / 80; G = 64 25 / 19,
// 37 / 46, 68 / 87; G = 32 29 / 20, 53 / 52, 102 / 96.  6 rows: G = 128 39 / 45, G = 64 48 / 48, G = 32 70 / 55.
inline bool experts_prefer_tiles(const LinearArgs& l, int sms, int mc) {
    const int active = std::min(l.R, l.E);
    const long long tiles = (long long)active * (l.ep.gated ? ceil_div(l.N / 2, 128) : ceil_div(l.N, kTcRows));
    if (2 * tiles < 3LL * sms) return false;               // (fewer tiles do not fill the SMs twice: another form)
    // experts of 8 rows on average take 1.5 sets each, of 4 rows one
    const double sets = active + std::max(0.0, (double)l.R / mc - 0.5 * active);
    const double units = sets * (l.ep.gated ? ceil_div(l.N / 2, 32) : ceil_div(l.N, 64));
    const double stage = l.G == 32 ? 1.75 : (l.G == 64 ? 1.13 : ((l.K / l.G) & 1 ? 1.17 : 0.87));
    const double decode = 8.0 + units / sms * std::max(1.2, stage * ceil_div(l.K, 1024));
    const double codes64 = l.G == 32 ? 0.78 : (l.G == 64 ? 0.70 : 0.66);
    return 9.0 + tiles / (2.0 * sms) * ceil_div(l.K, kGemmKB) * codes64 < decode;
}

// Which form takes a call.  The decode form takes up to 8 rows a matrix and whole 128-code blocks; above
// that the tensor-core tiles win.  A dense batch may also take two passes over the weights, which pays while
// the second comes from L2 and X leaves room for a ring: 16 rows x 4096, 28672 channels 26 us against 27 for
// the tiles, 4096 channels 8.6 against 9.8; 6 rows x 14336 17.4 against 19.8 (8 rows: 20.6 against 19.9).  It does
// not where weights are many (3 rows x 28672, 8192 channels: 61 against 43) or X is wide (16 rows x 14336: 33
// against 20).
inline awq_status launch_linear(const LinearArgs& l, const DeviceInfo& d, cudaStream_t st) {
    const int share = l.offsets ? ceil_div(l.R, std::min(l.R, l.E)) : l.R;
    // 64-row units where every CTA gets many (and a stage has 8 groups per row): half as many partial sums meet,
    // but the last round of units is twice as long.  Gated, pairs are counted, so the change comes at 16.  32-row
    // against 64-row units, us, 1 / 8 rows: 28672 x 4096 (6 a CTA) 15.1 / 17.6 against 15.4 / 18.2; 37888 x 4096 (8)
    // 17.6 / 20.8 against 17.1 / 20.1; 37888 x 2048, G = 64 13.5 / 16.7 against 12.8 / 13.6; 57344 x 4096 gated (12)
    // 24.4 / 28.5 against 24.6 / 29.0, 75776 x 4096 gated (16) 29.8 / 34.1 against 29.6 / 33.8; 3 rows each of 64 experts,
    // 2816 x 2048 gated (38) 58.9 against 39.4.  Below the limit 64 rows win at short K only: 18944 x 2048, G = 64 (4)
    // 8.7 / 10.9 against 8.4 / 9.4.
    const long long units = (long long)(l.offsets ? std::min(l.R, l.E) : 1) * ceil_div(l.ep.gated ? l.N / 2 : l.N, 32);
    const int RS = l.G <= 128 && units >= (long long)kDecManyUnits * d.sms ? 2 : 1;
    const int passes = l.offsets || share <= 1 || (long long)l.N * l.K > (128LL << 20) ? 1 : 2;
    if (share <= kDecMaxRows * passes && l.K % 128 == 0 && l.K <= kDecMaxK) {
        int mc = 0, S = 0;
        bool fits = dec_plan(l.R, l.K, l.G, RS, d.max_smem_optin, mc, S) && mc >= share;
        if (!fits && passes == 2)
            fits = dec_plan(ceil_div(share, 2), l.K, l.G, RS, d.max_smem_optin, mc, S) && 2 * mc >= share &&
                   (share <= kDecMaxRows || S >= 3);
        // a CTA's list of segments must hold the row sets that its units may reach
        const long long sets = !fits ? 0 : (l.offsets ? (long long)l.R / mc + std::min(l.R, l.E) : ceil_div(l.R, mc));
        if (fits && l.offsets && RS == 2 && experts_prefer_tiles(l, d.sms, mc)) fits = false;
        if (fits && sets <= (long long)(kDecMaxSegs - 2) * d.sms && sets * ceil_div(l.N, 32) < 0x7fffffffLL)
            return launch_linear_decode(l, d, RS, mc, S, st);
    }
    return launch_linear_tc(l, d.sms, st);
}

}  // namespace awq
