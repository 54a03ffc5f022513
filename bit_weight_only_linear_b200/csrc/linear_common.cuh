// Helpers shared by the fused and grouped linears, the routing and the combination: device primitives
// beside those of sm100.cuh, and the dependent launch.
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace awq {
namespace sm100 {

// True in one lane of a converged warp.  A branch on it tells the compiler that one thread runs
// what follows: tcgen05 and TMA instructions take their operands from uniform registers, and under
// a branch on the thread index the compiler wraps each in a loop over the active lanes (measured
// for tcgen05.mma of 128 rows: 189 cycles each whatever its N; elected, 9 at N = 16 and 96 at N = 192).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// mbar_wait for warps that must stay converged and cannot leave their loop on a time-out: a wait that
// runs out raises the timeout flag and sets *abort (shared memory), and every later wait that would block
// returns at once, so the loop runs out quickly (on data that the error word declares invalid).  The
// branches are inside the assembly: with the outcome tested outside, a wait on a phase that is already
// complete cost 140 cycles instead of 44 (the operands of the tensor-core instructions behind it have to
// go back to uniform registers), more than the MMAs of a k-block.
__device__ __forceinline__ void mbar_wait_or_abort(uint32_t bar, uint32_t parity, uint32_t abort) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u64 t0, t1;\n\t.reg .u32 f;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n\t"
        "@p bra DONE%=;\n\t"
        "mov.u64 t0, %%globaltimer;\n"
        "LOOP%=:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1, %3;\n\t"
        "@p bra DONE%=;\n\t"
        "ld.volatile.shared.u32 f, [%2];\n\t"
        "setp.ne.u32 q, f, 0;\n\t"
        "@q bra DONE%=;\n\t"
        "mov.u64 t1, %%globaltimer;\n\t"
        "sub.u64 t1, t1, t0;\n\t"
        "setp.lt.u64 q, t1, %4;\n\t"
        "@q bra LOOP%=;\n\t"
        "mov.u32 f, 1;\n\t"
        "st.volatile.shared.u32 [%2], f;\n\t"
        "red.global.or.b32 [%5], %6;\n"
        "DONE%=:\n\t}" ::"r"(bar),
        "r"(parity), "r"(abort), "r"(kWaitSuspendNs), "l"(kWaitLimitNs), "l"(__cvta_generic_to_global(&g_error_word)),
        "r"(kErrTimeout)
        : "memory");
}
__device__ __forceinline__ void mbar_wait_or_abort(uint64_t* bar, uint32_t parity, const volatile uint32_t* abort) {
    mbar_wait_or_abort(smem_u32(bar), parity, smem_u32(const_cast<const uint32_t*>(abort)));
}

// Wait until the stream's previous kernel has completed, then let the next one start.  In this order the
// next kernel's early reads (weights, in the decode form and the GEMV) come after everything before this one.
__device__ __forceinline__ void grid_dependency_pass() {
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

// 32 TMEM lanes x 8 consecutive 32-bit columns (as tmem_ld16).
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

}  // namespace sm100

// Launch as a programmatic dependent of the stream's previous kernel (every kernel launched so waits
// for it before it touches global memory).
inline bool launch_pdl(const void* fn, dim3 grid, dim3 block, void** args, cudaStream_t st) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = block;
    lc.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelExC(&lc, fn, args) == cudaSuccess;
}

}  // namespace awq
