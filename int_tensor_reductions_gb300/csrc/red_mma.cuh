// red_mma.cuh -- building blocks of matrix products on the tensor cores
// (tcgen05 with accumulators in tensor memory, operands staged by TMA): the
// instructions as functions, and the ring that feeds them.
//
// Two CTAs of a cluster work as a pair on one 256 x 256 tile (cta_group::2):
// each stages its 128 rows of A and its 128 columns' worth of B, the leader
// (rank 0) issues the products, and each CTA holds the accumulators of its
// 128 rows in its own tensor memory.  B crosses each SM's shared memory once
// for 256 rows; one CTA alone would read 48 KB of operands per 64 of K for
// half the work.
//
// An operand is staged as blocks of 128-byte rows with the 128-byte swizzle,
// in one of two orders, whichever lies contiguous in memory:
//   along K:      128 rows (of M or N) x 64 of K; a step of 16 of K is 32 bytes
//                 further, groups of 8 rows are 1024 bytes apart;
//   along M or N: blocks of 64 of K x 64 (of M or N), two for 128; a step of 16
//                 of K is 2048 bytes further, groups of 8 of K 1024 bytes and
//                 blocks 8192 bytes apart.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "red_pipeline.cuh"

namespace red {

constexpr int TILE = 256;             // rows and columns of a pair's tile
constexpr int HALF = TILE / 2;        // rows of A, and of B, that a CTA stages
constexpr int BLOCK_K = 64;           // 128 bytes of 16-bit elements
constexpr int OPERAND_BYTES = HALF * BLOCK_K * 2;
constexpr int STAGE_BYTES = 2 * OPERAND_BYTES;
constexpr int STAGES = 5;  // a sixth instead of the second box of each warp's results: the same (1907, 1883 TFLOP/s)

// ------------------------------------------------------------ instructions

// Shared-memory address of the same variable in the pair's leader.
__device__ __forceinline__ uint32_t leader_addr(const void *p)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_addr(p)));
    return a;
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// A box of a tensor map to this CTA's shared memory; its bytes count at `bar`,
// a barrier of either CTA of the pair (a cluster address).
__device__ __forceinline__ void tma_load(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap *map, int x, int y, const void *src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
                 "r"(y), "r"(smem_addr(src))
                 : "memory");
}
// As a store, adding to what is there (fp32, to nearest).
__device__ __forceinline__ void tma_add(const CUtensorMap *map, int x, int y, const void *src)
{
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
                 "r"(x), "r"(y), "r"(smem_addr(src))
                 : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Until all but N of this thread's groups of stores have read their shared memory /
// until all are written.
template <int N>
__device__ __forceinline__ void store_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Tensor memory of the pair: all 512 columns in each of its CTAs.  One warp of
// each CTA.
__device__ __forceinline__ void tmem_alloc(uint32_t *where)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(where)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(base) : "memory");
}
__device__ __forceinline__ void tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D (256 x 256, tensor memory) = or += A B^T over 16 of K.
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// Arrives at `bar` in both CTAs of the pair once the products so far are done.
__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// The same of one CTA alone: a tile of 128 rows.
__device__ __forceinline__ void tma_load_alone(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}
template <int COLUMNS>
__device__ __forceinline__ void tmem_alloc_alone(uint32_t *where)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "n"(COLUMNS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int COLUMNS>
__device__ __forceinline__ void tmem_free_alone(uint32_t base)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "n"(COLUMNS));
}
__device__ __forceinline__ void mma_alone(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_commit_alone(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// One lane of a warp (all of it calls), always the same.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
    return p != 0;
}

// Whether all lanes of a warp say so (WARP false: the one thread).
template <bool WARP = true>
__device__ __forceinline__ bool agreed(bool ok)
{
    return WARP ? __all_sync(0xffffffffu, ok) != 0 : ok;
}

// 16 columns of this warp's 32 lanes of tensor memory: lane i gets row i.
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ------------------------------------------------------------- descriptors

// Staged operand, 128-byte swizzle: start, stride between blocks of 64 of M or N
// (read along M or N only), 1024 bytes between groups of 8.
__device__ __forceinline__ uint64_t operand_desc(const void *p, bool along_k)
{
    return (uint64_t)((smem_addr(p) >> 4) & 0x3fffu) | (uint64_t)(along_k ? 1 : (8192 >> 4)) << 16 |
           (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// One step of 16 of K further, in the descriptor's units of 16 bytes.
__host__ __device__ constexpr uint64_t step_k(bool along_k) { return along_k ? 2 : 128; }

// f16 or bf16 operands, fp32 accumulators, a tile of rows x cols.
__device__ __forceinline__ uint32_t instruction_desc(bool bf16, bool a_along_k, bool b_along_k, int rows = TILE,
                                                     int cols = TILE)
{
    return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (a_along_k ? 0u : 1u << 15) | (b_along_k ? 0u : 1u << 16) |
           (uint32_t)(cols / 8) << 17 | (uint32_t)(rows / 16) << 24;
}

// ------------------------------------------------------------- the pipeline

struct MmaBarriers {
    uint64_t full[STAGES], empty[STAGES];  // operand stages; full: the leader's
    uint64_t acc_full[2], acc_empty[2];    // accumulators; empty: the leader's
    uint64_t drain;
    uint32_t tmem;
    int failed;
};

constexpr int MMA_THREADS = 384;   // warp 0: copies, 1: products, 2: tensor memory, 4 to 11: epilogue
constexpr int EPILOGUE_WARPS = 8;  // four groups of 32 rows times two halves of the columns
constexpr int BOX_BYTES = 4096;  // 32 rows of 128 bytes, two boxes per warp
constexpr int STAGING_BYTES = 2 * BOX_BYTES;
constexpr size_t MMA_SMEM = STAGES * STAGE_BYTES + EPILOGUE_WARPS * STAGING_BYTES + 1024;  // + alignment

// One tile's product: A rows from a_row, B rows from b_row (of M and N), `blocks`
// of 64 of K from a_k / b_k on.  Either operand may lie along K or along M / N
// (map: boxes of 64 x 128 or 64 x 64).
struct TileJob {
    const CUtensorMap *a, *b;
    int a_row, b_row, a_k, b_k;
    int blocks;
    bool a_along_k, b_along_k;
};

__device__ __forceinline__ void load_operand(unsigned char *dst, const CUtensorMap *map, int row, int k, bool along_k,
                                             uint32_t bar)
{
    if (along_k) {
        tma_load(dst, map, k, row, bar);
    } else {
        tma_load(dst, map, row, k, bar);
        tma_load(dst + OPERAND_BYTES / 2, map, row + 64, k, bar);
    }
}

// Ring positions that copies and products go through in the same order.
template <int N = STAGES>
struct RingPos {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++stage == N) {
            stage = 0;
            phase ^= 1;
        }
    }
};

// The copies of one tile (one thread of each CTA).  Whether to go on.
__device__ __forceinline__ bool copy_tile(const TileJob &j, MmaBarriers &b, unsigned char *ring, RingPos<> &pos, int rank)
{
    for (int k = 0; k < j.blocks; ++k) {
        if (!mbar_wait(&b.empty[pos.stage], pos.phase ^ 1, &b.failed, 0))
            return false;
        // the barrier of the leader takes the bytes of both
        if (rank == 0)
            mbar_expect(&b.full[pos.stage], 2 * STAGE_BYTES);
        const uint32_t bar = leader_addr(&b.full[pos.stage]);
        unsigned char *at = ring + pos.stage * STAGE_BYTES;
        load_operand(at, j.a, j.a_row + rank * HALF, j.a_k + k * BLOCK_K, j.a_along_k, bar);
        load_operand(at + OPERAND_BYTES, j.b, j.b_row + rank * HALF, j.b_k + k * BLOCK_K, j.b_along_k, bar);
        pos.next();
    }
    return true;
}

struct AccPos {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next()
    {
        slot ^= 1;
        phase ^= slot == 0;
    }
};

// The products of one tile (by the leading CTA), handed over after every `chunk` blocks of
// K, each time in the other accumulator.  Whether to go on.
// WARP: all lanes of a warp wait and one, the one that `issues` (elect_one()), issues: what the
// products take is then known to be the same for the warp, and one thread's moving it there
// takes as long as the products of a block (forward 6144 x 4096 x 65536 1775 -> 1662 us, 2777 x 1024 x 50257 168 -> 156).
// The lanes agree on each wait, one of which may have run out.  Else one thread calls.
template <bool WARP>
__device__ __forceinline__ bool multiply_tile(const TileJob &j, MmaBarriers &b, const unsigned char *ring, RingPos<> &pos,
                                              AccPos &acc, uint32_t idesc, int chunk, bool issues)
{
    const uint64_t ka = step_k(j.a_along_k), kb = step_k(j.b_along_k);
    for (int k0 = 0; k0 < j.blocks; k0 += chunk) {
        if (!agreed<WARP>(mbar_wait(&b.acc_empty[acc.slot], acc.phase ^ 1, &b.failed, 0)))
            return false;
        tmem_after();
        const uint32_t d = b.tmem + acc.slot * TILE;
        const int k1 = min(k0 + chunk, j.blocks);
        for (int k = k0; k < k1; ++k) {
            if (!agreed<WARP>(mbar_wait(&b.full[pos.stage], pos.phase, &b.failed, 0)))
                return false;
            tmem_after();
            const unsigned char *at = ring + pos.stage * STAGE_BYTES;
            const uint64_t da = operand_desc(at, j.a_along_k), db = operand_desc(at + OPERAND_BYTES, j.b_along_k);
            if (issues) {
#pragma unroll
                for (int s = 0; s < BLOCK_K / 16; ++s)
                    mma(d, da + s * ka, db + s * kb, idesc, k > k0 || s > 0);
                mma_commit(&b.empty[pos.stage]);
            }
            pos.next();
        }
        if (issues)
            mma_commit(&b.acc_full[acc.slot]);
        acc.next();
    }
    return true;
}

// Registers from the first four warps to the epilogue's eight, in a kernel
// launched with 168 per thread: 128 * 64 + 256 * 216 <= 384 * 168.
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 64;"); }
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 216;"); }

// Set-up and end of a kernel of pairs, by all threads.
__device__ __forceinline__ void mma_begin(MmaBarriers &b, int warp, int lane)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&b.full[i], 1);
            mbar_init(&b.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.acc_full[i], 1);
            mbar_init(&b.acc_empty[i], 2 * EPILOGUE_WARPS);
        }
        mbar_init(&b.drain, 1);
        b.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2)
        tmem_alloc(&b.tmem);
    tmem_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    tmem_after();
}
__device__ __forceinline__ void mma_end(MmaBarriers &b, int warp)
{
    tmem_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    tmem_after();
    if (warp == 2)
        tmem_free(b.tmem);
}

// What is left after a wait ran out: the copies and products in flight are
// waited for, within limits, before the CTA ends.
__device__ __forceinline__ void drain_copies(MmaBarriers &b, const RingPos<> &pos, int rank)
{
    if (rank == 0)
        for (int k = 0; k < STAGES; ++k)
            for (int n = 0; n < 65536 && !mbar_try(&b.full[k], k < pos.stage ? pos.phase : pos.phase ^ 1); ++n) {
            }
}
__device__ __forceinline__ void drain_products(MmaBarriers &b, bool issues)
{
    if (issues)
        mma_commit(&b.drain);
    for (int n = 0; n < 65536 && !mbar_try(&b.drain, 0); ++n) {
    }
}

}  // namespace red
