// Bounded waits on mbarriers, and the rings whose slots they guard.
#pragma once

#include "common.cuh"
#include "per_device.cuh"

namespace moedc {

constexpr unsigned long long kMvWaitNs = 200000000ull; // bound of every wait

__device__ __forceinline__ uint32_t smem_u32(const void* p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void mbar_init(uint64_t* b, int count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect(uint64_t* b, int bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t* b, int parity)
{
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n"
                 " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                 " selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok) : "r"(smem_u32(b)), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ unsigned long long globaltimer()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Bounded: false when the wait ran out or another one of the block did
// (*abort).  The callers then go on without waiting, so that every barrier of
// the block is still met and the kernel ends; the status word tells.
static __device__ __noinline__ bool mbar_wait_slow(uint64_t* b, int parity, volatile int* abort)
{
    // the timer is read only once the wait is a long one: reading it takes longer than
    // most waits
    unsigned long long t0 = 0;
    if (*abort) return false;
    for (int i = 0; ; ++i) {
        if (mbar_try(b, parity)) return true;
        if (i % 1024 != 1023) continue;
        if (*abort) return false;
        const unsigned long long now = globaltimer();
        if (t0 == 0) t0 = now;
        else if (now - t0 > kMvWaitNs) break;
    }
    *abort = 1;
    return false;
}
__device__ __forceinline__ bool mbar_wait(uint64_t* b, int parity, volatile int* abort)
{
    return mbar_try(b, parity) || mbar_wait_slow(b, parity, abort);
}

// The same without a call, for threads whose registers are full: what a call does not keep
// would be spilled around it.
__device__ __forceinline__ bool mbar_wait_inline(uint64_t* b, int parity, volatile int* abort)
{
    unsigned long long t0 = 0;
    for (int i = 1; !mbar_try(b, parity); ++i) {
        if (i % 1024 != 0) continue;
        const unsigned long long now = globaltimer();
        if (t0 == 0) t0 = now;
        if (*abort || now - t0 > kMvWaitNs) {
            *abort = 1;
            return false;
        }
    }
    return true;
}

// Where a stage's slot and phase go round the ring.
struct MvRing {
    int slot = 0, phase = 0;
    __device__ __forceinline__ void next(int stages)
    {
        if (++slot == stages) {
            slot = 0;
            phase ^= 1;
        }
    }
};

}  // namespace moedc

namespace moedc_host {

// `raised`: of this kernel
inline bool raise_smem_limit(PerDevice& raised, const void* kernel, int bytes)
{
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return false;
    return raised.once(device, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
    });
}

}  // namespace moedc_host
