// opt2s_mx4_wait.cuh -- waits on shared-memory barriers that give up.
//
// Nothing may hang: a wait is a limited number of attempts.  One that runs
// out raises its CTA's abort flag, at which the CTA's other waits end too, so
// that the CTA drains its copies, frees what it holds and returns.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace opt2s {
namespace {

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}

// Up to `limit` attempts; false when they ran out or the CTA is aborting.
// `errors` counts CTAs, so only the thread that raises the flag adds to it.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, uint32_t limit, volatile int* abort_flag,
                                         unsigned int* errors)
{
    for (uint32_t i = 0; i < limit; ++i) {
        if (bar_try(bar, parity)) return true;
        if ((i & 255u) == 255u && *abort_flag) return false;
    }
    if (atomicExch(const_cast<int*>(abort_flag), 1) == 0) atomicAdd(errors, 1u);
    return false;
}

}  // namespace
}  // namespace opt2s
