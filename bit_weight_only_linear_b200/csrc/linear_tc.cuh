// Fused linear and expert-grouped linear on the sm_100a tensor cores (tcgen05, TMA, TMEM),
// with the dequantised weights as the TMEM operand.
//
// D[n][m] = sum_k deq(W)[n][k] X[m][k]: a tile is 256 weight rows (two MMA row tiles of 128) by
// BN rows of X.  Gated, the two row tiles are 128 gate rows and the 128 rows F behind them, so
// that both halves of an output sit in one TMEM lane and the epilogue needs no exchange.
//
//   * A from tensor memory: a dequantising thread is one weight row = one TMEM lane; it turns
//     the row's packed codes into fp16 pairs and writes them with tcgen05.st.  Compared with an A
//     tile in shared memory this takes the 128 x 64 fp16 write and the MMA's reads of it off
//     shared memory, which at 128 B/cycle otherwise bounds the MMA: per 128 x BN x 16 MMA
//     (BN / 2 cycles) the shared memory then carries B (BN / 4 cycles), half of the copy of X
//     (BN / 8) and the packed words (16).
//   * B = X in the 128-byte-swizzled K-major layout, in a ring freed by the MMAs: by tiled TMA where
//     the rows are in place, by 16-byte cp.async where their numbers come from a table (the experts'
//     tokens; tile::gather4 took 37 cycles per four 128-byte rows whatever the number of issuing
//     warps, 0.7 of the rate below on a prefill).
//   * Packed weights: 256-code stages (a whole 128-byte line per row) in a ring of their own,
//     freed by the dequantisers.
//   * Few tiles: a cluster of `splits` CTAs shares the K of a tile; the fp32 partial sums meet in
//     distributed shared memory and are added in rank order (no workspace, no second kernel).
//   * Grouped: every expert's rows are cut into tiles of their own; a CTA finds its tile by a scan
//     over the offsets table, so nothing is read back to the host.
// Bound: the tensor cores from about 150 rows on (2048 rows x 57344 x 8192, gated: 1.32 to 1.34 ms in a short graph =
// 1430 to 1460 TFLOP/s, 0.87 of the measured burst rate; call after call, at the clocks the power cap leaves, 1.52 ms
// = 1270, 0.92 of the sustained rate); the round trip between conversion and MMA,
// 0.3 us per 64 codes of 256 rows, below (61 rows x 4096 x 14336: 24 us, of which 8 are the start and the
// exchange of the splits); with tiles of few rows the issue of the conversion (96 tokens, 6 of 64 experts,
// 2816 x 2048: 62 us = 3.2 TB/s).
// Each dequantised weight is rounded once to fp16, as in awq_linear_gemm, whose range flag it raises too: (q - z) *
// scale has 15 significant bits, the MMA's fp16 operand 11.  To keep them all would take a second MMA for the
// remainders, or unscaled codes as the operand and the 256 x BN sums read back and scaled after every group.  The
// error against 64 bits is 2.7e-4 (rms, relative; gated 3.3e-4), of which the output's own rounding is 2.1e-4; sums
// are fp32.  Every wait is bounded: on time-out the kernel raises the device error word, drains what it issued,
// frees TMEM and returns.
#pragma once

#include <algorithm>
#include <cmath>
#include <mutex>

#include "common.cuh"
#include "epilogue.cuh"
#include "gemm_sm100.cuh"
#include "gemv.cuh"
#include "launch.cuh"
#include "linear_common.cuh"
#include "sm100.cuh"

namespace awq {

// D[tmem] (+)= A[tmem] * B[smem desc]^T, kind::f16.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 TMEM lanes x 16 consecutive 32-bit columns, from registers.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One code pair of a word as fp16 1024 + q: (word & mask) | 0x6400 in both halves.  As one lop3: written in C it
// becomes two instructions, since each takes one immediate, and with 16 rows a tile the integer pipe's 9 per word
// instead of 5 were what the conversion waited for (96 tokens, 6 of 64 experts, 2816 x 2048: 71 -> 65 us).
__device__ __forceinline__ uint32_t code_pair(uint32_t word, uint32_t mask) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(word), "r"(mask), "r"(0x64006400u));
    return r;
}

// (q - z) * s for the 8 codes of a word, as 4 fp16 pairs in k order; the two codes of a pair sit at the same nibble
// of the word's halves.  q - z is exact, the product is rounded once.
__device__ __forceinline__ uint4 dequant_codes(uint32_t word, uint32_t zmagic, uint32_t zneg16, uint32_t s2) {
    uint32_t a = code_pair(word, 0x000F000Fu);             // 1024 + q
    uint32_t b = code_pair(word, 0x00F000F0u);             // 1024 + 16 q
    uint32_t c = code_pair(word >> 8, 0x000F000Fu);
    uint32_t d = code_pair(word >> 8, 0x00F000F0u);
    asm("sub.rn.f16x2 %0, %0, %4;\n\t"                     // less 1024 + z
        "sub.rn.f16x2 %2, %2, %4;\n\t"
        "fma.rn.f16x2 %1, %1, %5, %6;\n\t"                 // a sixteenth, less 64 + z
        "fma.rn.f16x2 %3, %3, %5, %6;\n\t"
        "mul.rn.f16x2 %0, %0, %7;\n\t"
        "mul.rn.f16x2 %1, %1, %7;\n\t"
        "mul.rn.f16x2 %2, %2, %7;\n\t"
        "mul.rn.f16x2 %3, %3, %7;"
        : "+r"(a), "+r"(b), "+r"(c), "+r"(d)
        : "r"(zmagic), "r"(0x2C002C00u), "r"(zneg16), "r"(s2));
    return make_uint4(a, b, c, d);
}

// 16 bytes global -> shared, or zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16u : 0u) : "memory");
}
// Arrive on `bar` once every cp.async of this thread so far has landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sm100::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Four fp32 at the shared-memory address `a` of this CTA, in CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_cluster4(uint32_t a, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .u32 r;\n\tmapa.shared::cluster.u32 r, %4, %5;\n\tld.shared::cluster.v4.f32 {%0, %1, %2, %3}, "
        "[r];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(a), "r"(rank)
        : "memory");
    return v;
}

constexpr int kTcMaxSplits = 8;          // CTAs of a cluster that share a tile's K
constexpr int kTcRows = 256;             // weight rows per tile: two MMA row tiles
constexpr int kTcWKB = 4;                // k-blocks (64 codes) per packed stage: 128-byte lines

template <int BN>
struct TcCfg {
    // Up to 64 columns two CTAs share an SM (8 dequantising warps, half of TMEM each): one's
    // start and epilogue overlap the other's stream.  Above, one CTA with 16 warps.
    static constexpr int kCtas = BN <= 64 ? 2 : 1;
    static constexpr int kDqWarps = BN <= 64 ? 8 : 16;
    static constexpr int kXWarps = BN == 16 ? 1 : 2;      // copy X (a gathered one; a tiled one takes a thread)
    static constexpr int kMmaWarp = kXWarps, kWWarp = kXWarps + 1, kDqWarp0 = kXWarps + 2;
    static constexpr int kThreads = 32 * (kDqWarp0 + kDqWarps);
    static constexpr uint32_t kTmemCols = 512 / kCtas;
    static constexpr int kABufs = BN == 128 ? 4 : 2;      // x 64 columns (two tiles x 64 codes); divides kTcWKB
    static constexpr int kXStages = BN == 192 ? 5 : (BN == 128 ? 6 : (BN == 64 ? 5 : (BN == 32 ? 10 : 6)));
    static constexpr int kWStages = BN == 64 || BN == 32 ? 2 : 3;
    static constexpr int kXBytes = BN * 128;
    static constexpr int kXBox = BN < 32 ? 16 : 32;                        // rows per copy of X
    static constexpr int kWBytes = kTcRows * 32 * kTcWKB;
    static constexpr int kWOff = 0;
    static constexpr int kXOff = kWOff + kWStages * kWBytes;
    static constexpr int kRing = kXOff + kXStages * kXBytes;
    static constexpr int kSrcOff = kRing;                                  // [BN] row numbers of X (negative: none)
    static constexpr int kBarOff = kSrcOff + BN * 4;
    static constexpr int kNumBars = 2 * kXStages + 2 * kWStages + 4 * kABufs + 1;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;                // TMEM address, tile, flags
    static constexpr int kSmemBytes = kMiscOff + 32 + 1024;
    static_assert(kSmemBytes <= (kCtas == 1 ? 232448 : 115712), "shared memory");
    static_assert(2 * BN + kABufs * 64 <= (int)kTmemCols, "tensor memory");
    static_assert(kTcRows * BN * 4 <= kRing, "the partial sums of a K split reuse the rings");
};

struct TcArgs {
    const uint16_t* X;
    long long ldx;                       // a multiple of 8
    const uint16_t* scales;
    const uint32_t* qzeros;              // NULL: implicit zero 8
    const int32_t* rows;                 // row numbers of X, or NULL
    const int32_t* offsets;              // [E+1], or NULL: one range of R rows
    int T, R, E, N, K;
    int n_tiles;                         // tiles of weight rows
    int m_tiles;                         // tiles of X rows (dense)
    int kb_per;                          // k-blocks per split (a multiple of kTcWKB)
    Epilogue ep;
};

// Row range of expert e, clamped into 0..R whatever the table holds.
__device__ __forceinline__ int2 expert_range(const int32_t* offsets, int e, int R) {
    const int b = min(max(__ldg(offsets + e), 0), R);
    return make_int2(b, min(max(__ldg(offsets + e + 1), b), R));
}

// Rows of each of the tiles of at most `bn` rows that `m` rows are cut into: even shares, in steps
// of `step` (a divisor of bn).
__device__ __forceinline__ int tile_rows(int m, int tiles, int step) {
    return ((m + tiles - 1) / tiles + step - 1) / step * step;
}

// The `tile`-th tile of the experts' ranges: {expert, first row, end of the tile's rows, tile of weight
// rows}, expert -1 if there are fewer tiles.  By a whole warp.  Each expert has ceil(rows / bn) row
// tiles by `per` tiles of weight rows, the row tiles innermost.
__device__ __forceinline__ int4 find_tile(const int32_t* offsets, int E, int R, int bn, int step, int per,
                                          long long tile) {
    const int lane = threadIdx.x & 31;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        int2 g = make_int2(0, 0);
        if (e < E) g = expert_range(offsets, e, R);
        const int mt = (g.y - g.x + bn - 1) / bn;
        long long x = (long long)mt * per, v = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        const long long total = __shfl_sync(0xffffffffu, x, 31);
        if (tile < total) {
            const bool mine = tile >= x - v && tile < x;
            const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
            const int in = (int)(tile - (x - v));          // tile inside the expert
            const int m = mt ? in % mt : 0, n = mt ? in / mt : 0;
            const int rows = mt ? tile_rows(g.y - g.x, mt, step) : 0;
            int4 r = make_int4(e, g.x + m * rows, min(g.y, g.x + (m + 1) * rows), n);
            r.x = __shfl_sync(0xffffffffu, r.x, src);
            r.y = __shfl_sync(0xffffffffu, r.y, src);
            r.z = __shfl_sync(0xffffffffu, r.z, src);
            r.w = __shfl_sync(0xffffffffu, r.w, src);
            return r;
        }
        tile -= total;
    }
    return make_int4(-1, 0, 0, 0);
}

template <int BN, int G>
__global__ void __launch_bounds__(TcCfg<BN>::kThreads, TcCfg<BN>::kCtas)
linear_tc_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_q,
                 const TcArgs a) {
    using C = TcCfg<BN>;
    using namespace sm100;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
    uint64_t* xfull = bars;                         // [kXStages] X landed
    uint64_t* xempty = xfull + C::kXStages;         // [kXStages] MMAs done with the slot
    uint64_t* wfull = xempty + C::kXStages;         // [kWStages] packed stage landed
    uint64_t* wempty = wfull + C::kWStages;         // [kWStages] dequantisers have read it
    uint64_t* afull = wempty + C::kWStages;         // [kABufs][2] dequantised k-block of a row tile in TMEM
    uint64_t* aempty = afull + 2 * C::kABufs;       // [kABufs][2] MMAs done with it
    uint64_t* tfull = aempty + 2 * C::kABufs;       // accumulators complete
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
    int32_t* src = reinterpret_cast<int32_t*>(smem + C::kSrcOff);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    uint32_t splits;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(splits));
    const uint32_t rank = cluster_rank();
    const int tile = blockIdx.x / splits;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kXStages; ++s) {
            mbar_init(&xfull[s], a.rows ? 32 * C::kXWarps : 1);
            mbar_init(&xempty[s], 1);
        }
        for (int s = 0; s < C::kWStages; ++s) {
            mbar_init(&wfull[s], 1);
            mbar_init(&wempty[s], C::kDqWarps);
        }
        for (int b = 0; b < 2 * C::kABufs; ++b) {
            mbar_init(&afull[b], C::kDqWarps / 2);
            mbar_init(&aempty[b], 1);
        }
        mbar_init(tfull, 1);
        mbar_fence_init();
        prefetch_tensormap(&tmap_x);
        prefetch_tensormap(&tmap_q);
    }
    if (warp == C::kMmaWarp) {
        tmem_alloc(&misc[0], C::kTmemCols);
        tmem_relinquish();
    }
    grid_dependency_pass();
    if (warp == 0) {
        // the CTA's tile and the rows of X that it reads
        int4 t;
        if (a.offsets)
            t = find_tile(a.offsets, a.E, a.R, BN, 16, a.n_tiles, tile);
        else {
            const int rows = tile_rows(a.R, a.m_tiles, 16), r0 = (tile % a.m_tiles) * rows;
            t = make_int4(0, r0, min(a.R, r0 + rows), tile / a.m_tiles);
        }
        if (t.y >= t.z) t.x = -1;
        if (lane == 0) {
            misc[1] = (uint32_t)t.x;
            misc[2] = (uint32_t)t.y;
            misc[3] = (uint32_t)t.z;
            misc[4] = (uint32_t)t.w;
        }
        if (t.x >= 0 && a.rows)
            for (int c = lane; c < BN; c += 32) {
                // (columns behind the tile's rows are never stored: any row does)
                const int s = __ldg(a.rows + min(t.y + c, t.z - 1));
                src[c] = s < a.T ? s : -1;
            }
        if (lane == 0) misc[5] = 0u;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    const int expert = (int)misc[1], r0 = (int)misc[2], r1 = (int)misc[3], nt = (int)misc[4];
    const int F = a.ep.gated ? a.N / 2 : a.N;
    // weight rows of the two row tiles inside the expert, and where they end
    const int n0 = a.ep.gated ? nt * 128 : nt * kTcRows;
    const int n1 = a.ep.gated ? F + n0 : n0 + 128;
    const int end0 = F, end1 = a.N;
    const int kb0 = rank * a.kb_per;
    const int num_kb = expert < 0 ? 0 : max(0, min(a.kb_per, ceil_div(a.K, kGemmKB) - kb0));
    const int n16 = (r1 - r0 + 15) & ~15;             // columns of the MMA: the tile's rows of X
    const int boxes = (n16 + C::kXBox - 1) / C::kXBox;
    const uint32_t acc0 = tmem, abase = tmem + 2 * BN;

    if (warp < C::kXWarps) {
        // ---------------- X ring ----------------
        if (a.rows) {
            // thread: 16-byte unit u of rows t0, t0 + kRowStep, ..; its arrival on the stage's barrier follows
            // when its copies have landed.  They are generic writes: the MMA's thread fences them (a fence
            // here would wait for the copies still under way).
            constexpr int kRowStep = C::kXWarps * 4, kRows = BN / kRowStep;
            const int u = threadIdx.x & 7, t0 = threadIdx.x >> 3;
            const int count = num_kb > 0 ? n16 / kRowStep : 0;          // rows of this thread
            uint32_t off[kRows];                                        // row starts in 16-byte units
            bool all = true;                                            // every row lies inside X
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int r = i < count ? src[t0 + i * kRowStep] : 0;
                all = all && r >= 0;
                off[i] = r < 0 ? 0xffffffffu : (uint32_t)((unsigned long long)r * (unsigned long long)(a.ldx >> 3));
            }
            all = __all_sync(0xffffffffu, all);
            const uint32_t dst0 = smem_u32(smem + C::kXOff) + (uint32_t)(t0 * 128 + ((u ^ (t0 & 7)) << 4));
            int s = 0;
            uint32_t ph = 0;
            for (int j = 0; j < num_kb; ++j) {
                mbar_wait_or_abort(&xempty[s], ph ^ 1u, &misc[5]);
                const int unit = (kb0 + j) * (kGemmKB / 8) + u;
                const uint4* base = reinterpret_cast<const uint4*>(a.X) + unit;
                const uint32_t dst = dst0 + (uint32_t)(s * C::kXBytes);
                const bool in_k = unit * 8 < a.K;
                if (all && __all_sync(0xffffffffu, in_k)) {
#pragma unroll
                    for (int i = 0; i < kRows; ++i) {
                        // (rows 4 apart: the swizzle follows row % 8)
                        const uint32_t flip = kRowStep % 8 ? (uint32_t)((i & 1) * 64) : 0u;
                        if (i < count) cp_async16((dst ^ flip) + (uint32_t)(i * kRowStep * 128), base + off[i], true);
                    }
                } else {
                    // zeros past K and for rows that do not exist
#pragma unroll 1
                    for (int i = 0; i < count; ++i) {
                        const uint32_t flip = kRowStep % 8 ? (uint32_t)((i & 1) * 64) : 0u;
                        const int r = src[t0 + i * kRowStep];
                        const bool live = in_k && r >= 0;
                        cp_async16((dst ^ flip) + (uint32_t)(i * kRowStep * 128),
                                   live ? a.X + r * a.ldx + unit * 8 : a.X, live);
                    }
                }
                cp_async_arrive(&xfull[s]);
                if (++s == C::kXStages) s = 0, ph ^= 1u;
            }
            cp_async_wait_all();        // before the CTA exits, or its ring is reused
        } else if (warp == 0 && elect_one()) {
            int issued = 0, s = 0;
            uint32_t ph = 0;
            for (int j = 0; j < num_kb; ++j) {
                if (!mbar_wait(&xempty[s], ph ^ 1u)) break;
                mbar_arrive_expect_tx(&xfull[s], (uint32_t)(boxes * C::kXBox * 128));
                for (int i = 0; i < boxes; ++i)
                    tma_load_2d(smem + C::kXOff + s * C::kXBytes + i * C::kXBox * 128, &tmap_x, &xfull[s],
                                (kb0 + j) * kGemmKB, r0 + i * C::kXBox);
                ++issued;
                if (++s == C::kXStages) s = 0, ph ^= 1u;
            }
            // every issued copy must land before the CTA may exit (or its ring be reused)
            for (int j = issued - 1; j >= 0 && j >= issued - C::kXStages; --j)
                mbar_wait(&xfull[j % C::kXStages], (j / C::kXStages) & 1);
        }
    } else if (warp == C::kWWarp) {
        if (elect_one()) {
            // ---------------- packed-weight ring ----------------
            const int n_st = ceil_div(num_kb, kTcWKB);
            int issued = 0, s = 0;
            uint32_t ph = 0;
            for (int j = 0; j < n_st; ++j) {
                if (!mbar_wait(&wempty[s], ph ^ 1u)) break;
                uint8_t* dst = smem + C::kWOff + s * C::kWBytes;
                const int x = (kb0 + j * kTcWKB) * (kGemmKB / 8);
                mbar_arrive_expect_tx(&wfull[s], C::kWBytes);
                tma_load_2d(dst, &tmap_q, &wfull[s], x, expert * a.N + n0);
                tma_load_2d(dst + C::kWBytes / 2, &tmap_q, &wfull[s], x, expert * a.N + n1);
                ++issued;
                if (++s == C::kWStages) s = 0, ph ^= 1u;
            }
            for (int j = issued - 1; j >= 0 && j >= issued - C::kWStages; --j)
                mbar_wait(&wfull[j % C::kWStages], (j / C::kWStages) & 1);
        }
    } else if (warp == C::kMmaWarp) {
        if (elect_one()) {
            // ---------------- MMA issuer ----------------
            const uint32_t idesc = idesc_f16_f32(128, n16);
            const uint64_t bdesc0 = desc_sw128_kmajor(smem_u32(smem + C::kXOff));
            int s = 0, b = 0;
            uint32_t xph = 0, aph = 0;
            for (int kb = 0; kb < num_kb; ++kb) {
                mbar_wait_or_abort(&xfull[s], xph, &misc[5]);
                if (a.rows) fence_proxy_async_smem();
                const uint64_t bdesc = bdesc0 + (uint64_t)(s * (C::kXBytes >> 4));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mbar_wait_or_abort(&afull[2 * b + h], aph, &misc[5]);
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kGemmKB / 16; ++kk)
                        mma_f16_ts(acc0 + h * BN, abase + (b * 2 + h) * 32 + kk * 8, bdesc + 2 * kk, idesc,
                                   (kb | kk) != 0);
                    mma_commit(&aempty[2 * b + h]);
                }
                mma_commit(&xempty[s]);
                if (++s == C::kXStages) s = 0, xph ^= 1u;
                if (++b == C::kABufs) b = 0, aph ^= 1u;
            }
            mma_commit(tfull);   // also on the error path, so that the MMAs drain before TMEM is freed
            mbar_wait(tfull, 0);
        }
    } else {
        // ---------------- dequantise: thread = weight row = TMEM lane ----------------
        constexpr int kSets = C::kDqWarps / 4;
        constexpr int kParts = 4 / kSets;         // 32-code halves of a k-block per thread: 1 or 2
        const int q = warp & 3;                   // TMEM lane quarter of this warp
        const int set = (warp - C::kDqWarp0) >> 2;
        const int h = set & 1;                    // row tile
        const int part0 = kParts == 1 ? set >> 1 : 0;
        const int r = q * 32 + lane;
        const int n = (h ? n1 : n0) + r;
        const bool row_ok = n < (h ? end1 : end0);
        const int ng = a.K / G;
        const int nzw = ceil_div(ng, 8);
        const bool zp = a.qzeros != nullptr;
        const size_t wrow = (size_t)max(expert, 0) * a.N + (row_ok ? n : 0);
        const uint16_t* srow = a.scales + wrow * ng;
        const uint32_t* zrow = a.qzeros + wrow * nzw;
        // scales and zeros of the stage's groups (256 / G, all in one zero word) are fetched a stage ahead;
        // with whole stages the scales are one aligned load
        constexpr int kGPS = 64 * kTcWKB / G;
        const bool whole = a.K % (64 * kTcWKB) == 0;
        uint32_t sc[(kGPS + 1) / 2] = {}, zw = 0x88888888u, sc_next[(kGPS + 1) / 2] = {}, zw_next = 0x88888888u;
        auto fetch = [&](int g0) {
            if (g0 >= ng) return;
            if (whole) {
                if constexpr (kGPS == 8) {
                    const uint4 t = __ldg(reinterpret_cast<const uint4*>(srow + g0));
                    sc_next[0] = t.x, sc_next[1] = t.y, sc_next[2] = t.z, sc_next[3] = t.w;
                } else if constexpr (kGPS == 4) {
                    const uint2 t = __ldg(reinterpret_cast<const uint2*>(srow + g0));
                    sc_next[0] = t.x, sc_next[1] = t.y;
                } else if constexpr (kGPS == 2) {
                    sc_next[0] = __ldg(reinterpret_cast<const uint32_t*>(srow + g0));
                } else {
                    sc_next[0] = __ldg(srow + g0);
                }
            } else {
#pragma unroll
                for (int i = 0; i < (kGPS + 1) / 2; ++i) {
                    sc_next[i] = g0 + 2 * i < ng ? __ldg(srow + g0 + 2 * i) : 0u;
                    if (kGPS > 1 && g0 + 2 * i + 1 < ng) sc_next[i] |= (uint32_t)__ldg(srow + g0 + 2 * i + 1) << 16;
                }
            }
            if (zp) zw_next = __ldg(zrow + (g0 >> 3));
        };
        int g0 = num_kb > 0 ? kb0 * kGemmKB / G : ng;
        fetch(g0);
        uint32_t s2 = 0, zmagic = 0x64006400u, zneg16 = 0, s_max = 0;
        // row r's line of a stage; its 16-byte unit u sits at u ^ (r % 8)
        const uint32_t wline = smem_u32(smem + C::kWOff) + (uint32_t)(h * (C::kWBytes / 2) + r * 128 + (r & 7) * 16);
        const uint32_t part_x = (uint32_t)(part0 * 16);
        const uint32_t aline = abase + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * 32 + part0 * 16);
        const uint32_t af = smem_u32(afull + h), ae = smem_u32(aempty + h), abort = smem_u32(&misc[5]);
        int ws = 0;
        uint32_t wph = 0, aph = 1;
#pragma unroll 1
        for (int kb = 0; kb < num_kb; kb += kTcWKB) {
            mbar_wait_or_abort(&wfull[ws], wph, &misc[5]);
            const uint32_t wr = (wline + ws * C::kWBytes) ^ part_x;
#pragma unroll
            for (int i = 0; i < (kGPS + 1) / 2; ++i) sc[i] = sc_next[i];
            zw = zw_next >> (4 * (g0 & 7));
            g0 += kGPS;
            fetch(g0);
            const int last = num_kb - kb;
#pragma unroll
            for (int sb = 0; sb < kTcWKB; ++sb) {
                if (sb >= last) break;
                constexpr int kBufMask = C::kABufs - 1;
                const int b = sb & kBufMask;
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                    const uint4 packed = lds128(wr ^ (uint32_t)(sb * 32 + i * 16));
                    // (G >= 64: both 32-code parts of a k-block are in one group; G = 32: one each)
                    const bool fresh = G == 32 || (i == 0 && (sb * 64) % G == 0);
                    if (fresh) {
                        uint32_t sg, z;
                        if constexpr (G == 32 && kParts == 1) {
                            sg = part0 ? sc[sb] >> 16 : sc[sb] & 0xFFFFu;
                            z = (zw >> (8 * sb + 4 * part0)) & 15u;
                        } else {
                            const int gi = (sb * 64 + i * 32) / G;
                            sg = gi & 1 ? sc[gi >> 1] >> 16 : sc[gi >> 1] & 0xFFFFu;
                            z = (zw >> (4 * gi)) & 15u;
                        }
                        s2 = sg * 0x00010001u;
                        zmagic = 0x64006400u + z * 0x00010001u;              // 1024 + z
                        zneg16 = 0xD400D400u + z * 0x00100010u;              // -(64 + z)
                        s_max = max(s_max, sg);
                    }
                    uint32_t v[16];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t word = w == 0 ? packed.x : (w == 1 ? packed.y : (w == 2 ? packed.z : packed.w));
                        const uint4 d = dequant_codes(word, zmagic, zneg16, s2);
                        v[4 * w] = d.x, v[4 * w + 1] = d.y, v[4 * w + 2] = d.z, v[4 * w + 3] = d.w;
                    }
                    // the codes are converted before the wait for the MMAs that read this buffer
                    if (i == 0) {
                        // use number (kb + sb) / kABufs of the buffer
                        const uint32_t parity = C::kABufs == kTcWKB ? aph : (uint32_t)(((sb / C::kABufs) & 1) ^ 1);
                        mbar_wait_or_abort(ae + b * 16, parity, abort);
                        __syncwarp();
                        tc_fence_after();
                    }
                    tmem_st16(aline + (uint32_t)(b * 64 + i * 16), v);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(af + b * 16) : "memory");
            }
            aph ^= 1u;
            if (lane == 0) mbar_arrive(&wempty[ws]);
            if (++ws == C::kWStages) ws = 0, wph ^= 1u;
        }
        // 15 scale16 may pass fp16 from 0x6C44 (4368) on (a negative scale or NaN counts as large here):
        // then every group of the row is looked at
        if (s_max >= 0x6C44u && row_ok) {
            const int g1 = min(ng, ceil_div((kb0 + num_kb) * kGemmKB, G));
            for (int g = kb0 * kGemmKB / G; g < g1; ++g) {
                const uint32_t z = zp ? (__ldg(zrow + (g >> 3)) >> (4 * (g & 7))) & 15u : 8u;
                const float sf = fabsf(h2f(__ldg(srow + g)));
                if (!(sf * (zp ? fmaxf((float)z, 15.0f - (float)z) : 8.0f) < 65520.0f) && !isnan(sf)) raise_error(kErrRange);
            }
        }
        const bool ok = __all_sync(0xffffffffu, num_kb > 0 && mbar_wait(tfull, 0) && misc[5] == 0);
        tc_fence_after();

        // ---------------- epilogue ----------------
        const Epilogue& ep = a.ep;
        const uint16_t* bias = ep.bias ? ep.bias + (size_t)max(expert, 0) * a.N : nullptr;
        if (splits == 1) {
            if (ok) {
                // gated: a warp takes both accumulators of its lanes and 1/kSets of the columns;
                // else one accumulator and 2/kSets of the columns
                const int hh = set & 1;
                const int cw = ep.gated ? BN / kSets : BN * 2 / kSets;
                const int c0 = ep.gated ? set * cw : (set >> 1) * cw;
                const int nn = (ep.gated ? n0 : (hh ? n1 : n0)) + r;
                const bool out_ok = nn < (ep.gated ? F : a.N);
                const float b0 = bias && out_ok ? h2f(bias[nn]) : 0.0f;
                const float b1 = bias && out_ok && ep.gated ? h2f(bias[F + nn]) : 0.0f;
                constexpr int CH = BN / kSets < 16 ? 8 : 16;          // columns at a time
                const uint32_t at = acc0 + (ep.gated ? 0 : hh * BN) + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
                for (int c = c0; c < c0 + cw && r0 + c < r1; c += CH) {
                    uint32_t u0[CH], u1[CH];
                    if constexpr (CH == 16) {
                        tmem_ld16(at + c, u0);
                        if (ep.gated) tmem_ld16(at + BN + c, u1);
                    } else {
                        tmem_ld8(at + c, u0);
                        if (ep.gated) tmem_ld8(at + BN + c, u1);
                    }
                    const int nv = out_ok ? min(CH, r1 - r0 - c) : 0;       // columns to store
                    float res[CH];
                    if (ep.residual) {
                        const uint16_t* rp = ep.residual + (size_t)(r0 + c) * ep.ldr + nn;
#pragma unroll
                        for (int i = 0; i < CH; ++i) {
                            res[i] = i < nv ? h2f(*rp) : 0.0f;
                            rp += ep.ldr;
                        }
                    }
                    tmem_ld_wait();
                    float y[CH];
#pragma unroll
                    for (int i = 0; i < CH; ++i) y[i] = __uint_as_float(u0[i]) + b0;
                    apply_act(y, ep.act);
                    if (ep.gated) {
#pragma unroll
                        for (int i = 0; i < CH; ++i) y[i] *= __uint_as_float(u1[i]) + b1;
                    }
                    if (ep.residual) {
#pragma unroll
                        for (int i = 0; i < CH; ++i) y[i] += res[i];
                    }
                    uint16_t* yp = ep.Y + (size_t)(r0 + c) * ep.ldy + nn;
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        if (i < nv) *yp = f2h_rn(y[i]);
                        yp += ep.ldy;
                    }
                }
            }
        } else if (ok) {
            // partial sums into this CTA's shared memory: [column][256 rows]
            float* part = reinterpret_cast<float*>(smem);
            const uint32_t lanes = (uint32_t)(q * 32) << 16;
            constexpr int cw = BN * 2 / kSets;
            constexpr int CH = cw < 16 ? 8 : 16;
            const int c0 = (set >> 1) * cw;
            for (int c = c0; c < c0 + cw && r0 + c < r1; c += CH) {
                uint32_t u[CH];
                if constexpr (CH == 16) tmem_ld16(acc0 + h * BN + lanes + (uint32_t)c, u);
                else tmem_ld8(acc0 + h * BN + lanes + (uint32_t)c, u);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < CH; ++i) part[(c + i) * kTcRows + h * 128 + r] = __uint_as_float(u[i]);
            }
        } else {
            float* part = reinterpret_cast<float*>(smem);
            // no k-block of this split (or a time-out, which is flagged): it adds nothing
            for (int i = threadIdx.x - 32 * C::kDqWarp0; i < kTcRows * BN; i += 32 * C::kDqWarps) part[i] = 0.0f;
        }
    }
    if (splits > 1) {
        __syncwarp();
        cluster_sync_all();
        // rank's share of the outputs: columns rank, rank + splits, ..; a thread takes four weight rows of a
        // column and adds the partial sums in rank order, all reads under way at once
        const uint32_t base = smem_u32(smem);
        const Epilogue& ep = a.ep;
        const int quads = ep.gated ? 32 : kTcRows / 4;
        const int cols = expert < 0 ? 0 : r1 - r0;
        const int mine = cols > (int)rank ? (cols - 1 - (int)rank) / (int)splits + 1 : 0;
        const uint16_t* bias = ep.bias ? ep.bias + (size_t)max(expert, 0) * a.N : nullptr;
        for (int i = threadIdx.x; i < mine * quads; i += C::kThreads) {
            const int c = (int)rank + (i / quads) * (int)splits, l = (i % quads) * 4;
            const int nn = n0 + l;                 // (not gated: n1 = n0 + 128)
            if (nn >= F) continue;
            const size_t m = r0 + c;
            float v[2][4] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h && !ep.gated) break;
                const uint32_t at = base + (uint32_t)(c * kTcRows + h * 128 + l) * 4;
                float4 p[kTcMaxSplits];
#pragma unroll
                for (int s = 0; s < kTcMaxSplits; ++s)
                    if (s < (int)splits) p[s] = ld_cluster4(at, (uint32_t)s);
#pragma unroll
                for (int s = 0; s < kTcMaxSplits; ++s)
                    if (s < (int)splits) v[h][0] += p[s].x, v[h][1] += p[s].y, v[h][2] += p[s].z, v[h][3] += p[s].w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (bias && nn + j < F) {
                    v[0][j] += h2f(bias[nn + j]);
                    if (ep.gated) v[1][j] += h2f(bias[F + nn + j]);
                }
            apply_act(v[0], ep.act);
            uint16_t* yp = ep.Y + m * ep.ldy + nn;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (nn + j >= F) break;
                float y = v[0][j];
                if (ep.gated) y *= v[1][j];
                if (ep.residual) y += h2f(ep.residual[m * ep.ldr + nn + j]);
                yp[j] = f2h_rn(y);
            }
        }
        __syncwarp();
        cluster_sync_all();     // no CTA leaves while another reads its shared memory
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// Copies the rows of X that the experts' rows name (zeros for numbers outside X) into `out` [R][K], so
// that the tiles can read them in place.  A warp per row and pass; rows that no expert owns are left.
constexpr int kGatherThreads = 256;

__global__ void __launch_bounds__(kGatherThreads)
gather_rows_kernel(const uint16_t* __restrict__ X, int T, long long ldx, const int32_t* __restrict__ rows, int R,
                   const int32_t* __restrict__ offsets, int E, int K, uint16_t* __restrict__ out) {
    sm100::grid_dependency_pass();
    const int lane = threadIdx.x & 31;
    const int begin = min(max(__ldg(offsets), 0), R), end = min(max(__ldg(offsets + E), 0), R);
    for (long long p = begin + (long long)blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5); p < end;
         p += (long long)gridDim.x * (kGatherThreads / 32)) {
        const int r = __ldg(rows + p);
        const bool live = r >= 0 && r < T;
        const uint4* src = reinterpret_cast<const uint4*>(X + (live ? r : 0) * ldx);
        uint4* dst = reinterpret_cast<uint4*>(out + p * K);
#pragma unroll 4
        for (int i = lane; i < K / 8; i += 32) dst[i] = live ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Rows per expert from which a gathered product first copies its rows in order: the copy costs 4 R K
// bytes and a launch, the gathering producers hold the MMAs up (4096 tokens x 2 of 8 experts, 28672 x 4096:
// 1758 us gathered in place, 1530 copied first; 64 rows an expert 253 and 211).
constexpr int kGatherMinShare = 64;

inline size_t gather_workspace_bytes(int R, int E, int K) {
    if (R <= 0 || E <= 0 || K <= 0 || (long long)R < (long long)kGatherMinShare * E) return 0;
    return align256((size_t)R * K * 2);
}

struct LinearArgs {
    const uint16_t* X;
    int T;                       // rows of X
    long long ldx;
    const int32_t* rows;         // row numbers of X per output row, or NULL
    int R;                       // output rows
    const int32_t* offsets;      // [E+1] or NULL (dense: one range of R rows)
    int E;
    const uint32_t* qweight;
    const uint16_t* scales;
    const uint32_t* qzeros;      // NULL: implicit zero 8
    int N, K, G;
    Epilogue ep;
    void* ws;                    // gather_workspace_bytes(), or NULL: rows are gathered in place
    size_t ws_bytes;
};

inline bool make_tmap_ld(CUtensorMap* map, const void* base, CUtensorMapDataType dtype, uint64_t rows, uint64_t cols,
                         uint64_t row_bytes, uint32_t box_rows, uint32_t box_cols) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {row_bytes};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, dtype, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, int G>
awq_status launch_tc(const LinearArgs& l, int splits, cudaStream_t st) {
    using C = TcCfg<BN>;
    CUtensorMap tx, tq;
    if (!make_tmap_ld(&tx, l.X, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (uint64_t)l.T, (uint64_t)l.K, (uint64_t)l.ldx * 2,
                      C::kXBox, kGemmKB))
        return AWQ_ERR_CUDA;
    if (!make_tmap_ld(&tq, l.qweight, CU_TENSOR_MAP_DATA_TYPE_UINT32, (uint64_t)l.E * l.N, (uint64_t)(l.K / 8),
                      (uint64_t)l.K / 2, 128, kTcWKB * kGemmKB / 8))
        return AWQ_ERR_CUDA;
    const void* fn = (const void*)linear_tc_kernel<BN, G>;
    if (!prepare_kernel(fn)) return AWQ_ERR_CUDA;
    TcArgs a = {l.X, l.ldx, l.scales, l.qzeros, l.rows, l.offsets, l.T, l.R, l.E, l.N, l.K, 0, 0, 0, l.ep};
    a.n_tiles = l.ep.gated ? ceil_div(l.N / 2, 128) : ceil_div(l.N, kTcRows);
    a.m_tiles = ceil_div(l.R, BN);
    const int num_kb = ceil_div(l.K, kGemmKB);
    a.kb_per = ceil_div(ceil_div(num_kb, splits), kTcWKB) * kTcWKB;
    if (l.rows && (unsigned long long)l.T * (unsigned long long)(l.ldx >> 3) >= 0xffffffffull) return AWQ_ERR_UNSUPPORTED;
    // grouped: the experts that have rows add at most one partial tile each
    const long long mt = l.offsets ? (long long)l.R / BN + std::min(l.R, l.E) : a.m_tiles;
    const long long ctas = mt * a.n_tiles * splits;
    if (ctas > 0x7fffffffLL) return AWQ_ERR_UNSUPPORTED;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)ctas);
    lc.blockDim = dim3(C::kThreads);
    lc.dynamicSmemBytes = C::kSmemBytes;
    lc.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 2;
    void* args[] = {&tx, &tq, &a};
    return cudaLaunchKernelExC(&lc, fn, args) == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

template <int BN>
awq_status launch_tc_bn(const LinearArgs& l, int splits, cudaStream_t st) {
    switch (l.G) {
        case 32: return launch_tc<BN, 32>(l, splits, st);
        case 64: return launch_tc<BN, 64>(l, splits, st);
        case 128: return launch_tc<BN, 128>(l, splits, st);
        default: return launch_tc<BN, 256>(l, splits, st);
    }
}

// Clusters of `splits` CTAs that can be resident at once on the current device, per kernel (a driver
// query, made once: the GPU's processing clusters do not divide evenly; of 8 CTAs with one on each SM, a
// B200 holds 15 clusters, of 6 CTAs 22, of 4 CTAs 33).
template <int BN>
int tc_active_clusters(int splits) {
    using C = TcCfg<BN>;
    static std::mutex mu;
    static int known[64][kTcMaxSplits + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lk(mu);
    int& n = known[dev][splits];
    if (n == 0) {
        const void* fn = (const void*)linear_tc_kernel<BN, 128>;
        if (!prepare_kernel(fn)) return 0;
        cudaLaunchConfig_t lc = {};
        lc.gridDim = dim3((unsigned)splits);
        lc.blockDim = dim3(C::kThreads);
        lc.dynamicSmemBytes = C::kSmemBytes;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)splits;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        lc.attrs = attr;
        lc.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, fn, &lc) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = -1;
        }
    }
    return n;
}

// Modelled time (us) of `tiles` tiles of `rows` rows of X with the K in `splits` parts, from measured
// slopes: a k-block of 256 weight rows takes 0.30 us, or 3.5 ns per row of X (0.38 and 3.0 in the 192-row form;
// 24 rows measure 0.31, 61 0.37, 96 0.45, 192 0.67, with the HBM's share where all SMs stream); a
// tile 4 us (6) around them, and 7 (12) for the exchange of a split's partial sums.  A last partial wave
// costs half of one on average.
template <int BN>
double tc_time(long long tiles, int rows, int num_kb, int splits) {
    const int active = tc_active_clusters<BN>(splits);
    if (active < 1) return 1e30;
    const int kb = ceil_div(ceil_div(num_kb, splits), kTcWKB) * kTcWKB;
    double waves = (double)tiles / active;
    waves = waves <= 1.0 ? 1.0 : std::min(std::ceil(waves), waves + 0.5);
    double t = kb * (BN == 192 ? std::max(0.38, 0.0030 * rows) : std::max(0.30, 0.0035 * rows)) + (BN == 192 ? 6.0 : 4.0);
    if (splits > 1) t += BN == 192 ? 12.0 : 7.0;
    return waves * t;
}

inline awq_status launch_linear_tc(const LinearArgs& l, int sms, cudaStream_t st) {
    // rows to plan for: the dense batch, or the experts' average share with a margin for uneven ones
    const int active = l.offsets ? std::min(l.R, l.E) : 1;
    const int m = l.offsets ? (int)std::min<long long>(l.R, ((long long)l.R * 13 + active * 10 - 1) / (active * 10)) : l.R;
    const int n_tiles = l.ep.gated ? ceil_div(l.N / 2, 128) : ceil_div(l.N, kTcRows);
    const int num_kb = ceil_div(l.K, kGemmKB);
    // Few rows and many tiles: two CTAs on an SM hide each other's start and end (64 experts of 9 rows, 2816 x
    // 2048: 62 us at 32 rows a tile against 92 with one CTA; with fewer tiles than SMs it is the reverse,
    // 16 tiles of 61 rows x 14336 in 6 parts: 24 us against 28).  A tile holds 2.2 times the experts' average,
    // since a second tile reads an expert's weights again (the same experts at tiles of 16 / 32 / 64 rows, 6 rows
    // each: 61 / 62 / 65 us, 9: 65 / 62 / 65, 12: 69 / 63 / 66, 16: 78 / 67 / 67, 19: 87 / 71 / 67).  Skewed shares, 9 rows
    // on average: one expert with 96 62 us, two with 96 68; 8 on average: one with 256 of 512 rows 70.
    if (m <= 64 && 2LL * active * n_tiles >= 3LL * sms) {
        const long long hold = l.offsets ? ((long long)l.R * 11 + active * 5 - 1) / (active * 5) : l.R;
        if (hold <= 16) return launch_tc_bn<16>(l, 1, st);
        if (hold <= 32) return launch_tc_bn<32>(l, 1, st);
        return launch_tc_bn<64>(l, 1, st);
    }
    LinearArgs in_place = l;
    if (l.rows && l.offsets && l.ws) {
        const size_t need = gather_workspace_bytes(l.R, l.E, l.K);
        if (need && l.ws_bytes >= need) {
            uint16_t* out = static_cast<uint16_t*>(l.ws);
            void* args[] = {&in_place.X, &in_place.T, &in_place.ldx, &in_place.rows, &in_place.R,
                            &in_place.offsets, &in_place.E, &in_place.K, &out};
            const long long blocks = std::min<long long>(8LL * sms, ceil_div(l.R, kGatherThreads / 32));
            if (!launch_pdl((const void*)gather_rows_kernel, dim3((unsigned)blocks), dim3(kGatherThreads), args, st))
                return AWQ_ERR_CUDA;
            in_place.X = out;
            in_place.T = l.R;
            in_place.ldx = l.K;
            in_place.rows = nullptr;
        }
    }
    int best = 1;
    bool wide = false;
    double best_t = 1e30;
    for (int w = 0; w < 2; ++w) {
        const int mt = ceil_div(m, w ? 192 : 128), rows = (ceil_div(m, mt) + 15) & ~15;
        const long long tiles = (long long)active * mt * n_tiles;
        for (int s = 1; s <= kTcMaxSplits && (s == 1 || num_kb >= 4 * s); ++s) {
            const double t = w ? tc_time<192>(tiles, rows, num_kb, s) : tc_time<128>(tiles, rows, num_kb, s);
            if (t < best_t) best_t = t, best = s, wide = w;
        }
    }
    return wide ? launch_tc_bn<192>(in_place, best, st) : launch_tc_bn<128>(in_place, best, st);
}

}  // namespace awq
