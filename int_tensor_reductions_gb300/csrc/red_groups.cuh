// red_groups.cuh -- rows held in the registers of a group of lanes: loads and
// stores of 16 bytes per lane, reductions over the group, and the group that a
// row's length asks for.  8 to 32 lanes of a warp, or a whole CTA, hold a row;
// unit u of lane l is the E elements (16 bytes) from (u * LANES + l) * E on.  (Eight
// consecutive fp32 values per lane would be two loads of every other 16 bytes:
// norm 16384 x 4096 f32 231 us, as it is 173.)
#pragma once

#include <cstdint>
#include <type_traits>

#include "red_internal.h"
#include "red_loss.cuh"
#include "red_pipeline.cuh"

namespace red {

// Threads of a CTA: one group, or several in 256.
template <int LANES>
constexpr int GROUP_CTA = LANES > 32 ? LANES : 256;

// ------------------------------------------------------------- row access

// Elements of a unit, and units of a lane that holds `VECS` times eight elements.
template <int DT>
constexpr int UNIT = DT == RED_F32 ? 4 : 8;
template <int DT, int VECS>
constexpr int UNITS = VECS * 8 / UNIT<DT>;

// A unit as it lies in memory.
struct Raw {
    uint32_t u[4];
};

template <int DT>
__device__ __forceinline__ void widen(const Raw &r, float (&v)[UNIT<DT>])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (DT == RED_F32) {
            v[k] = __uint_as_float(r.u[k]);
        } else {
            v[2 * k] = Elem<DT>::widen(r.u[k] & 0xffffu);
            v[2 * k + 1] = Elem<DT>::widen(r.u[k] >> 16);
        }
    }
}
template <int DT>
__device__ __forceinline__ Raw narrow(const float (&v)[UNIT<DT>])
{
    Raw r;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (DT == RED_F32)
            r.u[k] = __float_as_uint(v[k]);
        else
            r.u[k] = (uint32_t)Elem<DT>::narrow(v[2 * k]) | (uint32_t)Elem<DT>::narrow(v[2 * k + 1]) << 16;
    }
    return r;
}

// The first n elements of a unit, one by one; 0 behind them.
template <int DT>
__device__ __forceinline__ Raw load_some(const void *p, int64_t at, int n)
{
    Raw r;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (DT == RED_F32) {
            r.u[k] = k < n ? static_cast<const uint32_t *>(p)[at + k] : 0u;
        } else {
            const uint16_t *q = static_cast<const uint16_t *>(p) + at;
            r.u[k] = (2 * k < n ? (uint32_t)q[2 * k] : 0u) | (2 * k + 1 < n ? (uint32_t)q[2 * k + 1] << 16 : 0u);
        }
    }
    return r;
}

// A lane's units of a row (`row`: the row's first element); 0 behind its end.
// The loads are issued together: nothing here looks at what they bring.
template <int DT, bool VEC, int LANES, int N>
__device__ __forceinline__ void load_row(Raw (&r)[N], const void *p, int64_t row, int lane, int len)
{
    constexpr int E = UNIT<DT>;
    if constexpr (VEC) {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int i = (u * LANES + lane) * E;
            const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const char *>(p) + (row + i) * (16 / E));
            const uint4 x = i + E <= len ? *q : make_uint4(0, 0, 0, 0);
            r[u].u[0] = x.x, r[u].u[1] = x.y, r[u].u[2] = x.z, r[u].u[3] = x.w;
        }
        if (len % E == 0)
            return;
    }
    // elements one by one: of one lane's last unit, or of all
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int i = (u * LANES + lane) * E;
        if (!VEC || (i < len && i + E > len))
            r[u] = load_some<DT>(p, row + i, len - i);
    }
}

template <int DT, bool VEC>
__device__ __forceinline__ void store_unit(void *p, int64_t row, int i, int len, const float (&v)[UNIT<DT>])
{
    constexpr int E = UNIT<DT>;
    if (VEC && i + E <= len) {
        const Raw r = narrow<DT>(v);
        *reinterpret_cast<uint4 *>(static_cast<char *>(p) + (row + i) * (16 / E)) =
            make_uint4(r.u[0], r.u[1], r.u[2], r.u[3]);
        return;
    }
#pragma unroll
    for (int k = 0; k < E; ++k)
        if (i + k < len)
            store_elem<DT>(p, row + i + k, v[k]);
}

// ------------------------------------------------------- rows fetched ahead

__device__ __forceinline__ void fetch16(void *dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fetch_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A ring of rows in shared memory, fetched while earlier rows are at work: each
// thread fetches its own units of ARRAYS matrices and reads them back itself, so
// that no barrier is needed.  Only rows on 16-byte boundaries go this way (VEC);
// others are loaded when they are wanted.
template <int DT, int LANES, int N, int ARRAYS>
struct Ring {
    static constexpr int NT = GROUP_CTA<LANES>;
    static constexpr int STAGE = ARRAYS * N * NT * 16;
    // one row at work, one on its way; more are no use (norm 30000 x 512 bf16 with four 18.4 us, with two 17.3)
    static constexpr int STAGES = 2 * STAGE <= 204800 ? 2 : 1;
    static constexpr size_t BYTES = (size_t)STAGE * STAGES;

    static __device__ __forceinline__ uint4 *slot(unsigned char *ring, int stage, int array, int u)
    {
        return reinterpret_cast<uint4 *>(ring) + ((stage * ARRAYS + array) * N + u) * NT + threadIdx.x;
    }
    static __device__ __forceinline__ void fetch(unsigned char *ring, int stage, int array, const void *p, int64_t row,
                                                 int lane, int len)
    {
        constexpr int E = UNIT<DT>;
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int i = (u * LANES + lane) * E;
            const int left = (len - i) * (16 / E);
            const uint32_t bytes = left <= 0 ? 0 : left < 16 ? left : 16;
            fetch16(slot(ring, stage, array, u), static_cast<const char *>(p) + (bytes ? (row + i) * (16 / E) : 0), bytes);
        }
    }
    static __device__ __forceinline__ Raw take(unsigned char *ring, int stage, int array, int u)
    {
        const uint4 x = *slot(ring, stage, array, u);
        return {{x.x, x.y, x.z, x.w}};
    }
};

// ------------------------------------------------------------ group reduction

template <int LANES>
struct GroupShared {
    float part[2][LANES / 32];
};
template <>
struct GroupShared<8> {
};
template <>
struct GroupShared<16> {
};
template <>
struct GroupShared<32> {
};

// The fold of v over a group, in every lane of it.  `turn` alternates from call to
// call, which saves the second barrier of a CTA-wide one.
template <int LANES, class F>
__device__ __forceinline__ float group_fold(float v, GroupShared<LANES> &sh, int &turn, F f)
{
#pragma unroll
    for (int o = (LANES < 32 ? LANES : 32) / 2; o; o >>= 1)
        v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    if constexpr (LANES > 32) {
        constexpr int WARPS = LANES / 32;
        if (threadIdx.x % 32 == 0)
            sh.part[turn][threadIdx.x / 32] = v;
        __syncthreads();
        v = sh.part[turn][threadIdx.x % WARPS];
#pragma unroll
        for (int o = WARPS / 2; o; o >>= 1)
            v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
        turn ^= 1;
    }
    return v;
}

struct Add {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {  // NaN wins
    __device__ __forceinline__ float operator()(float a, float b) const
    {
        float r;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
        return r;
    }
};

// Sums over the CTAs of a cluster of what each has in `share` (n floats in shared
// memory at the same place; all threads): f(i, sum) for this CTA's part of 0..n, in a
// fixed order.  One CTA alone goes through all of it.
template <class F>
__device__ __forceinline__ void cluster_sums(float *share, int n, F f)
{
    const int ctas = cluster_size(), rank = cluster_rank();
    __syncthreads();
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
    }
    for (int i = rank * blockDim.x + threadIdx.x; i < n; i += ctas * blockDim.x) {
        float sum = 0.0f;
        for (int c = 0; c < ctas; ++c)
            sum += *in_cta(share + i, c);
        f(i, sum);
    }
    if (ctas > 1) {  // (shared memory lives until the others have read it)
        cluster_arrive();
        cluster_wait();
    }
}

// The group of a row of `vecs` vectors (up to 2048).  Calls f with (lanes,
// vectors per lane).
template <class F>
int with_group(int vecs, F f)
{
    using std::integral_constant;
#define RED_GROUP(l, v) f(integral_constant<int, l>(), integral_constant<int, v>())
    if (vecs <= 8)
        return RED_GROUP(8, 1);
    if (vecs <= 16)
        return RED_GROUP(16, 1);
    if (vecs <= 32)
        return RED_GROUP(32, 1);
    if (vecs <= 64)
        return RED_GROUP(32, 2);
    if (vecs <= 128)
        return RED_GROUP(32, 4);
    if (vecs <= 256)
        return RED_GROUP(128, 2);
    if (vecs <= 384)
        return RED_GROUP(128, 3);
    if (vecs <= 512)
        return RED_GROUP(256, 2);
    if (vecs <= 768)
        return RED_GROUP(256, 3);
    if (vecs <= 1024)
        return RED_GROUP(256, 4);
    if (vecs <= 1536)
        return RED_GROUP(512, 3);
    return RED_GROUP(512, 4);
#undef RED_GROUP
}

// Whether a matrix's rows start on 16-byte boundaries (NULL: there is none).
inline bool aligned_rows(const void *p, int64_t ld, int64_t rows, int elem)
{
    return !p || ((uintptr_t)p % 16 == 0 && (rows < 2 || ld * elem % 16 == 0));
}

// CTAs per SM of a kernel, per device.
struct Resident {
    std::atomic<int> per_sm[64] = {};
};

// CTAs of a persistent grid: what is resident at once, or what there is to do; at most `most`.
template <class K>
int resident_grid(K kernel, Resident &cache, int threads, size_t smem, int64_t ctas, int64_t most, unsigned *grid)
{
    DeviceInfo di;
    const int st = device_info(&di);
    if (st != RED_OK)
        return st;
    int per_sm = cache.per_sm[di.dev].load(std::memory_order_relaxed);
    if (per_sm == 0) {
        cudaError_t e = cudaSuccess;
        if (smem > 0)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, (const void *)kernel, threads, smem);
        if (e != cudaSuccess)
            return cuda_fail(e, "occupancy");
        per_sm = per_sm > 0 ? per_sm : 1;
        cache.per_sm[di.dev].store(per_sm, std::memory_order_relaxed);
    }
    int64_t cap = (int64_t)per_sm * di.sms;
    cap = cap < most ? cap : most;
    *grid = (unsigned)(ctas < cap ? ctas : cap);
    return RED_OK;
}

}  // namespace red
