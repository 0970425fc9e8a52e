// red_pipeline.cuh -- barriers of asynchronous copies with waits of limited
// length, and clusters of CTAs.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace red {

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint64_t *bar, int count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(smem_addr(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}

// No wait is without end.  One that runs out, after `limit` tries in vain (0:
// after 20 s, which takes a hardware fault), marks the CTA as failed; what it
// has not written by then becomes NaN.
struct Patience {
    unsigned limit;
    unsigned tries = 0;
    uint64_t since = 0;

    __device__ __forceinline__ explicit Patience(unsigned n) : limit(n) {}
    static __device__ __forceinline__ uint64_t now()
    {
        uint64_t t;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        return t;
    }
    // After a try in vain: whether to give up.
    __device__ __forceinline__ bool spent(volatile int *failed)
    {
        ++tries;
        if (limit != 0) {
            if (tries < limit && !*failed)
                return false;
        } else {
            if (tries % 256 != 0)
                return false;
            if (tries == 256)
                since = now();
            if (!*failed && now() - since < 20000000000ull)
                return false;
        }
        *failed = 1;
        return true;
    }
};

// Whether the phase was over before the wait ran out.
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, volatile int *failed, unsigned limit)
{
    if (mbar_try(bar, parity))
        return true;
    Patience patience(limit);
    while (!mbar_try(bar, parity))
        if (patience.spent(failed))
            return false;
    return true;
}

// ---- clusters

__device__ __forceinline__ int cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return (int)r;
}
__device__ __forceinline__ int cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return (int)r;
}
// The same shared variable in CTA `rank` of the cluster.
template <class V>
__device__ __forceinline__ V *in_cta(V *p, int rank)
{
    uint64_t d;
    asm volatile("mapa.u64 %0, %1, %2;" : "=l"(d) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
    return reinterpret_cast<V *>(d);
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

}  // namespace red
