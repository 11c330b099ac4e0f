// What the tensor-core kernels of the draft step share beyond kda_sm100.cuh.
#pragma once

#include "kda_common.cuh"
#include "kda_sm100.cuh"

namespace kda {

constexpr uint64_t kDraftWaitNs = 2000000000ull;

// A bounded wait on an mbarrier.  A thread that gave up reports it and does not wait again: it
// goes through the rest of its schedule at once (its other barriers, which count threads, still
// see it), so that no other thread waits for it beyond its own bound.
struct Waiter {
    int* status;
    bool alive = true;
    __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity)
    {
        if (!alive) return;
        if (sm100::mbar_try_wait(bar, parity)) return;
        const uint64_t t0 = sm100::globaltimer_ns();
        while (!sm100::mbar_try_wait_sleep(bar, parity, 1000)) {
            if (sm100::globaltimer_ns() - t0 > kDraftWaitNs) {
                alive = false;
                report_status(status, kDevTimeout);
                return;
            }
        }
    }
};

// barrier `id` over `threads` threads of the block (whole warps)
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// 2^x, to 2 ulp (subnormal results become zero)
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace kda
