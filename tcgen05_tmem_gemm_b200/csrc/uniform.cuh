// Roles that run as whole warps.  The tensor core's and the copy engine's
// instructions take their operands from uniform registers.  In a branch of one
// lane the compiler has to move each operand there for each instruction: about
// 118 cycles between two tcgen05 instructions, measured with %clock64, where an
// MMA of 256 x 256 x 16 takes 128 and a copy of scales far less.  So the warp
// that issues them runs its loop with all lanes, on values that are the same in
// every lane by construction, and only the instruction itself belongs to one.
#pragma once

#include "sm100.cuh"

namespace dg {

// One lane of a whole warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// A value that every lane has, in a form the compiler knows to be uniform.
__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

// mbar_wait by a whole warp; false, in every lane, when one gave up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtl &w) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, w));
}

// Arrive on an mbarrier of another CTA of the cluster once this thread's TMEM
// loads are done (tcgen05.wait::ld, then the fence).  Not a release to the
// cluster (mbar_arrive_cluster): nothing in memory is handed over, and one would
// wait for every store of C before it, 3000 cycles at the end of a tile.
__device__ __forceinline__ void mbar_arrive_tmem(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

}  // namespace dg
