// What the tensor-core kernels of the draft step share beyond kda_sm100.cuh.
#pragma once

#include "kda_common.cuh"
#include "kda_sm100.cuh"

namespace kda {

constexpr uint64_t kDraftWaitNs = 2000000000ull;

// A bounded wait on an mbarrier: one test in line, then a loop of a handful of instructions.
// The roles of a kernel share its instruction cache, so what is in line at every wait counts:
// with a clock read and the report there tree_decode took 234 us instead of 228 (64 x 96 heads x
// 16 nodes), and with the first test inside the loop's block the attention took 272 us
// instead of 267 (32 trees of 16 nodes).  It gives up after 2^20 suspensions of about a
// microsecond.  A thread that gave up does not wait again: it goes through the rest of its
// schedule at once (its other barriers, which count threads, still see it), so that no other
// thread waits for it beyond its own bound; the owner calls finish() at the end, which reports it.
struct Waiter {
    int* status;
    bool alive = true;
    __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity)
    {
        if (!alive || sm100::mbar_try_wait(bar, parity)) return;
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .u32 n;\n\t"
            "mov.u32 n, 1048576;\n"
            "again:\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
            "@p bra done;\n\t"
            "sub.u32 n, n, 1;\n\t"
            "setp.ne.u32 p, n, 0;\n\t"
            "@p bra again;\n"
            "done:\n\t"
            "min.u32 %0, n, 1;\n\t}"
            : "=r"(ok)
            : "r"(sm100::smem_u32(bar)), "r"(parity)
            : "memory");
        alive = ok != 0;
    }
    __device__ __forceinline__ void finish() const
    {
        if (!alive) report_status(status, kDevTimeout);
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
