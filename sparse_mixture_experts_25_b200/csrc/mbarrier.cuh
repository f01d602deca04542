// Shared-memory mbarriers, bounded waits on them and untiled bulk copies, for
// the kernels that stream rows through a ring of shared-memory stages (the
// tensor-map GEMMs keep their own wrappers beside their tile code).
#pragma once

#include "moe_internal.cuh"

namespace moe {

// a wait that lasts longer gives up, records DEVERR_TIMEOUT and leaves
constexpr unsigned long long kTimeoutNs = 2000000000ull;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
}

__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Warp-collective bounded wait: true when the phase with `parity` completed;
// false on abort (flag raised elsewhere) or timeout (raises the flag and records
// it).  Every lane returns the same result.  The timer
// is read only once a wait has gone on for a while: reading %globaltimer costs
// far more than a wait that is already over.
__device__ __forceinline__ bool warp_wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                  unsigned long long* counters) {
    const uint32_t a = smem_u32(bar);
    const int lane = threadIdx.x & 31;
    unsigned long long t0 = 0;
    for (uint32_t it = 0;; ++it) {
        if (__all_sync(0xffffffffu, mbar_try_wait(a, parity))) return true;
        if ((it & 63u) == 63u) {
            int stop = 0;
            if (lane == 0) {
                const unsigned long long now = global_timer_ns();
                if (t0 == 0) t0 = now;
                if (*abort_flag) {
                    stop = 1;
                } else if (now - t0 > kTimeoutNs) {
                    *abort_flag = 1;
                    atomicOr(counters + CNT_DEVICE_ERROR, (unsigned long long)DEVERR_TIMEOUT);
                    stop = 1;
                }
            }
            if (__shfl_sync(0xffffffffu, stop, 0)) return false;
        }
    }
}

// One thread's copy of `bytes` (a multiple of 16) from global to this CTA's
// shared memory, both 16-byte aligned, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// orders this thread's generic accesses of shared memory before later copies
// by the async proxy into it
__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

}  // namespace moe
