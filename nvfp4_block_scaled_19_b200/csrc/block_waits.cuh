// Shared memory, mbarriers and bounded waits of the kernels around a projection
// (residual_norm.cu, lora_tile.cu), and of their self-test (block_api.cu).  The
// GEMM's, which set the error word in its own translation unit, are in ptx.cuh.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "nvfp4.h"

namespace nvfp4 {

constexpr uint64_t kBlockTimeoutNs = 2000000000ull;

__device__ __forceinline__ uint32_t s32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t timer_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}

// The initialised barriers, before threads or copies use them.
__device__ __forceinline__ void bar_init_fence() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Where a wait that gives up says so.
struct Abort {
    volatile int *flag;  // shared, seen by every role
    int *err;            // the library's device error word
    uint64_t limit_ns = kBlockTimeoutNs;
};

// Waits for the phase with this parity.  Gives up, and returns false, when another
// thread of the CTA has, or after the limit: then it records the timeout and says
// so to the others.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, const Abort &ab, int tag) {
    if (bar_try(bar, parity)) return true;
    uint64_t t0 = 0;
    while (!*ab.flag) {
        // The clock that bounds the wait is slow to read: between many tries.
#pragma unroll 1
        for (int i = 0; i < 256; ++i)
            if (bar_try(bar, parity)) return true;
        const uint64_t now = timer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > ab.limit_ns) {
            if (atomicCAS(&ab.err[0], 0, NVFP4_ERR_TIMEOUT) == 0) ab.err[1] = tag;
            *ab.flag = 1;
        }
    }
    return false;
}

// The same by a whole warp: lane 0 polls, so the warp cannot part.
__device__ __forceinline__ bool bar_wait_warp(uint32_t bar, uint32_t parity, const Abort &ab, int tag) {
    int ok = 0;
    if ((threadIdx.x & 31) == 0) ok = bar_wait(bar, parity, ab, tag) ? 1 : 0;
    return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

// On the way out after a timeout: waits for copies or MMAs in flight, bounded.
__device__ __forceinline__ void bar_drain(uint32_t bar, uint32_t parity, uint64_t deadline) {
    while (!bar_try(bar, parity))
        if (timer_ns() > deadline) return;
}

__device__ __forceinline__ uint4 ld_shared_16B(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

}  // namespace nvfp4
