// sv_async.cuh -- barriers in shared memory with bounded waits, and TMA copies of page
// boxes, for the attention kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#ifdef __CUDACC__
namespace sv {

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t* b, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(b)), "r"(parity)
        : "memory");
    return ok;
}
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// without the hardware's own patience
__device__ __forceinline__ bool bar_test(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(b)), "r"(parity)
        : "memory");
    return ok;
}
// False once the wait has run out, here or (dead) in another warp of the CTA.  A limit
// below the device timer's tick means one look.  (The timer is slow to read: only after
// many tries.)
__device__ __forceinline__ bool bar_wait_long(uint64_t* b, uint32_t parity, unsigned long long limit, volatile int* dead) {
    unsigned long long t0 = 0;
    for (uint32_t i = 0; limit >= 1000; ++i) {
        if (bar_try(b, parity)) return true;
        if (*dead) return false;
        if ((i & 255u) == 255u) {
            const unsigned long long t = now_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 >= limit) break;
        }
    }
    *dead = 1;
    return false;
}
// by a whole warp, with one answer
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, unsigned long long limit, volatile int* dead) {
    if (__all_sync(0xFFFFFFFFu, bar_test(b, parity))) return true;
    return __all_sync(0xFFFFFFFFu, bar_wait_long(b, parity, limit, dead));
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// a box of a page's rows, for one head: `part` (64 elements), row, head, page
__device__ __forceinline__ void tma_part(uint32_t dst, const CUtensorMap* map, int part, int row, int head, int page,
                                         uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2,%3,%4,%5,%6}], [%7];" ::"r"(dst),
        "l"(map), "r"(0), "r"(row), "r"(part), "r"(head), "r"(page), "r"(smem_u32(bar))
        : "memory");
}
// a box of a page's rows of codes, for one head: row, head, page
__device__ __forceinline__ void tma_codes(uint32_t dst, const CUtensorMap* map, int row, int head, int page,
                                          uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2,%3,%4,%5}], [%6];" ::"r"(dst),
        "l"(map), "r"(0), "r"(row), "r"(head), "r"(page), "r"(smem_u32(bar))
        : "memory");
}
// all parts of the rows, one part after the other
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int row, int head, int page,
                                        uint64_t* bar) {
    tma_part(dst, map, 0, row, head, page, bar);
}

}  // namespace sv
#endif  // __CUDACC__
