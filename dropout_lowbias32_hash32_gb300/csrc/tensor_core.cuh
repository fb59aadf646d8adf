// tensor_core.cuh -- the sm_103a instructions that the attention kernels are
// built on, as inline PTX: mbarriers with bounded waits, TMA tile loads,
// tensor memory (TMEM) and tcgen05.mma.
#pragma once

#include <cuda.h>

#include <cstdint>
#include <type_traits>

#include "barrier.cuh"
#include "element.cuh"

namespace rngk {

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

// A value that all lanes of the warp have, for the compiler to know it: what
// follows from it is computed once a warp.
template <class T>
__device__ __forceinline__ T uniform(T v)
{
    return __shfl_sync(0xFFFFFFFFu, v, 0);
}

// ---- TMA ------------------------------------------------------------------------

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z, int32_t u, int32_t v)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], [%2];"
        ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v)
        : "memory");
}
// ---- work from blocks that have not started ------------------------------------------
// A running block takes over the work of one that the launch still has to
// start (cluster launch control): 16 bytes of answer to `response`, counted by
// the barrier.  After an answer that there is none, nobody asks again.
__device__ __forceinline__ void ask_for_work(uint32_t response, uint32_t bar)
{
    barrier_expect(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 ::"r"(response), "r"(bar)
                 : "memory");
}
// The index of the block whose work was taken over; -1 for none.
__device__ __forceinline__ int32_t taken_work(uint32_t response)
{
    int32_t taken, index;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.s32 %0, 1, 0, p;\n\t"
        "mov.b32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, r;\n\t}"
        : "=r"(taken), "=r"(index)
        : "r"(response)
        : "memory");
    return taken ? index : -1;
}

// A block's items of work: its own first, then those of blocks that need not
// start any more.  Every role goes through them.  The loading role asks for the
// next one when it has asked for all of an item's tiles, not before: an item
// that is taken too early waits while blocks that have finished go without.
struct WorkQueue {
    uint32_t response, answered, heard;  // shared-memory addresses: 16 bytes, and two barriers
    volatile uint32_t *stalled;
    uint32_t items = 0;

    // The next item, for a whole warp; -1 when there is none, or after a wait
    // that ran out.
    __device__ __forceinline__ int32_t next_warp()
    {
        if (!barrier_wait(answered, items++ & 1u, stalled)) return -1;
        const int32_t next = taken_work(response);
        fence_async_shared();
        __syncwarp();
        if (elect_one()) barrier_arrive(heard);
        return uniform(next);
    }
    // The loading role's: asks, once all others have heard the last answer.
    __device__ __forceinline__ int32_t ask_warp()
    {
        if (items && !barrier_wait(heard, (items - 1) & 1u, stalled)) return -1;
        if (elect_one()) ask_for_work(response, answered);
        if (!barrier_wait(answered, items & 1u, stalled)) {
            barrier_drain(answered, items & 1u);
            return -1;
        }
        ++items;
        return taken_work(response);
    }
};

// ---- a launch that may begin under the one before it -----------------------------------
// The next launch's blocks may start as soon as every block of this one has
// said so and there is room; they wait for this one's end, and see its writes,
// at grid_wait.
__device__ __forceinline__ void grid_let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A named barrier of kThreads threads; all_of also tells whether every one of
// them agrees.
template <int kThreads>
__device__ __forceinline__ void sync_threads(int id)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kThreads) : "memory");
}
template <int kThreads>
__device__ __forceinline__ bool all_of(int id, bool agree)
{
    uint32_t yes;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, %2, %3, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(yes)
        : "r"(static_cast<uint32_t>(agree)), "r"(id), "n"(kThreads)
        : "memory");
    return yes != 0;
}

// ---- tensor memory ---------------------------------------------------------------
// 512 columns of 128 lanes x 32 bits; an address is lane << 16 | column.  A warp
// reaches the 32 lanes of its rank in its group of four.

template <uint32_t kColumns>
__device__ __forceinline__ void tmem_alloc(uint32_t result)  // by a whole warp; writes the address to shared memory
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(result), "n"(kColumns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <uint32_t kColumns>
__device__ __forceinline__ void tmem_free(uint32_t address)  // by a whole warp
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(address), "n"(kColumns) : "memory");
}

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 (or 16, 8) adjacent columns of the warp's lanes, a lane to a thread.
__device__ __forceinline__ void tmem_load(uint32_t (&r)[32], uint32_t address)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(address));
}
__device__ __forceinline__ void tmem_load(uint32_t (&r)[16], uint32_t address)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(address));
}
// Ends the warp's loads so far; the registers pass through it, so that nothing
// that uses them moves ahead of it.
template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 16)
        asm volatile(""
                     : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]),
                       "+r"(r[i + 7]), "+r"(r[i + 8]), "+r"(r[i + 9]), "+r"(r[i + 10]), "+r"(r[i + 11]), "+r"(r[i + 12]),
                       "+r"(r[i + 13]), "+r"(r[i + 14]), "+r"(r[i + 15]));
}
template <int... N>
__device__ __forceinline__ void tmem_wait_load(uint32_t (&...r)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    (pin(r), ...);
}
__device__ __forceinline__ void tmem_store(uint32_t address, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
        ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
          "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
          "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
          "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(address)
        : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t address, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
        ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
          "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(address)
        : "memory");
}

__device__ __forceinline__ void tmem_store(uint32_t address, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};"
                 ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(address)
                 : "memory");
}

// ---- tcgen05.mma -------------------------------------------------------------------
// Operand tiles in shared memory are rows of 64 16-bit elements (128 bytes, a
// TMA box with the 128-byte swizzle; 1024-byte aligned), 8 rows to a swizzle
// atom.  With the product's inner index along the row ("row-major"), a step of
// 16 is 32 bytes into the row and atoms follow each other every 1024 bytes.
// With it across the rows ("column-major": the tile is used transposed), a step
// of 16 is 16 rows, and the next 64 of the outer index are `chunk` bytes on.

constexpr uint64_t kDescriptorBase = (uint64_t(1) << 46)     // descriptor version of sm_100 and later
                                     | (uint64_t(2) << 61);  // 128-byte swizzle

__device__ __forceinline__ uint64_t row_major_tile(uint32_t address)
{
    return kDescriptorBase | ((address >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32);
}
__device__ __forceinline__ uint64_t column_major_tile(uint32_t address, uint32_t chunk)
{
    return kDescriptorBase | ((address >> 4) & 0x3FFFu) | (uint64_t((chunk >> 4) & 0x3FFFu) << 16) |
           (uint64_t(1024 >> 4) << 32);
}

// How far step i of 16 is into a row-major tile of boxes, as a descriptor counts.
__host__ __device__ constexpr uint32_t row_step(int i, uint32_t box) { return (i / 4 * box + i % 4 * 32) / 16; }

// 16-bit operands of type T, f32 accumulators, M = 128 rows by N columns.
template <class T>
__host__ __device__ constexpr uint32_t mma_shape(uint32_t n, bool b_column_major)
{
    const uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    return (1u << 4) | (type << 7) | (type << 10) | ((b_column_major ? 1u : 0u) << 16) | ((n >> 3) << 17) |
           ((128u >> 4) << 24);
}

// D (+)= A B^T for one step of 16, A in shared memory or in TMEM (two elements
// to a column).  By one thread.
__device__ __forceinline__ void mma_step(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(shape), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}
__device__ __forceinline__ void mma_step_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t shape, bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(shape), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}
// Arrives at the barrier when every tcgen05 operation that this thread issued
// so far has completed.
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// A warpgroup's registers a thread; all four warps, and the block's shares add
// up to at most what it was launched with.
template <int kRegisters>
__device__ __forceinline__ void take_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegisters));
}
template <int kRegisters>
__device__ __forceinline__ void give_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegisters));
}

// ---- arithmetic ---------------------------------------------------------------------

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

}  // namespace rngk
