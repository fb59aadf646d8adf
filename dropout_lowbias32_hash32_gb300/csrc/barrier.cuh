// barrier.cuh -- mbarriers with bounded waits, and the bulk copies that they
// count, as inline PTX.
#pragma once

#include <cstdint>

namespace rngk {

// Waits that ran out in this translation unit's kernels (rng_debug_stalled_waits).
static __device__ unsigned long long g_stalled_waits;

__device__ __forceinline__ uint32_t smem_address(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---- mbarriers ----------------------------------------------------------------

__device__ __forceinline__ void barrier_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool barrier_try(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(2000)  // suspended for 2 us at most
        : "memory");
    return done != 0;
}

// Waits for the phase of the given parity to end, about two seconds at most;
// false when that ran out.  `stalled` (shared by the block) then makes every
// later wait return false at once: the block issues nothing more, waits for
// what it has in flight, frees what it holds and ends, and the host can read
// that it happened.  barrier_wait is for a whole warp, which it leaves
// converged; barrier_wait_one for a single thread.
__device__ __forceinline__ bool barrier_wait_one(uint32_t bar, uint32_t parity, volatile uint32_t *stalled)
{
#pragma unroll 1
    for (uint32_t tries = 0; !barrier_try(bar, parity); ++tries) {
        if (*stalled) return false;
        if (tries == 1u << 20) {
            *stalled = 1;
            atomicAdd(&g_stalled_waits, 1ull);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool barrier_wait(uint32_t bar, uint32_t parity, volatile uint32_t *stalled)
{
    return __all_sync(0xFFFFFFFFu, barrier_wait_one(bar, parity, stalled));
}
// The end of a block's role that gave up: waits, with a limit, for a phase.
__device__ __forceinline__ void barrier_drain(uint32_t bar, uint32_t parity)
{
#pragma unroll 1
    for (uint32_t tries = 0; tries < 100000 && !barrier_try(bar, parity); ++tries) {}
}

__device__ __forceinline__ void fence_barrier_init() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
// Orders this thread's shared-memory writes before later asynchronous reads.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// bytes adjacent bytes, a multiple of 16 from a 16-byte boundary to one.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

}  // namespace rngk
