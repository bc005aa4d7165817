// sm100_grouped_ptx.cuh -- PTX wrappers that the grouped products use besides those of
// sm100_ptx.cuh.  Like there, each is a direct statement of an instruction.
#pragma once

#include "sm100_ptx.cuh"

namespace forge {

// Barrier `id` (1..15; 0 is __syncthreads) among `threads` threads of the block.
__device__ __forceinline__ void named_barrier_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The same barrier; true for everyone if `ok` was true for everyone.
__device__ __forceinline__ bool named_barrier_all(int id, int threads, bool ok) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "bar.red.and.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(id), "r"(threads), "r"((uint32_t)ok)
        : "memory");
    return all != 0;
}

// 3-D tiled store shared -> global (what lies outside the tensor is not written).
__device__ __forceinline__ void tma_store_3d(const void* map, const void* smem_src, int c0, int c1,
                                             int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
            map),
        "r"(smem_u32(smem_src)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// Waits until this thread's bulk stores have been written.
__device__ __forceinline__ void tma_store_wait_all() {
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

}  // namespace forge
