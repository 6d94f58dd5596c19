// tc_issue.cuh -- device helpers of the kernels whose warps have roles of their own: copies by
// three-dimensional tensor maps, one elected lane, bounded waits by polls, register splits.
#pragma once

#include <stdint.h>

#include "umma.cuh"

namespace dr {
namespace tc {

using namespace umma;

__device__ __forceinline__ void tma_load_3d(void *dst, const void *tmap, uint64_t *bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(smem_u32(dst)), "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2) : "memory");
}
__device__ __forceinline__ void tma_store_3d(const void *tmap, const void *src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(tmap), "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2) : "memory");
}
__device__ __forceinline__ float ex2(float x) {   // 2^x, two ulp; 0 below the normal range
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// One lane of a whole warp.  The compiler knows that this is one, and takes the operands of the MMAs
// and copies behind it as they are; behind `lane == 0` it wraps each in a search for equal lanes
// (forward of B8 T4096 H16 d128 144 us instead of 121).
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
    return e != 0;
}
// The rest of a wait that was not over at once: at most *polls more polls (each of 60 cycles at
// least: a thirtieth of a second in all); then *polls becomes 0 and nobody waits any more.  Few
// instructions, for the many places that wait, and no call: the register split rules calls out.
constexpr int kPolls = 1 << 20;
__device__ __forceinline__ void wait_longer(uint64_t *bar, uint32_t parity, volatile int *polls) {
    int i = 0;
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if (++i > *polls) {
            *polls = 0;
            break;
        }
    }
}

template <int N>
__device__ __forceinline__ void more_regs() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_regs() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace tc
}  // namespace dr
