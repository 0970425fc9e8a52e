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

// Rows that start anywhere (on an element): 16-byte blocks of memory are read and
// written whole and their bytes moved in registers.  `off` is a row's distance from
// the block it starts in, the same for all its units.  A block that a row shares
// with what lies before or behind it is read whole, too (it is one transaction, and
// never crosses into memory that no allocation holds), and written by elements.
// (Element by element, norm 8000 x 4095 bf16: 192 us, as it is 79.)
__device__ __forceinline__ int block_offset(const void *p) { return (int)((uintptr_t)p & 15); }

// 16 bytes from byte `off` of the 32 in lo, hi on.
template <int DT>
__device__ __forceinline__ Raw window(const uint4 &lo, const uint4 &hi, int off)
{
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const bool by2 = off & 8, by1 = off & 4;
#pragma unroll
    for (int k = 0; k < 6; ++k)
        w[k] = by2 ? w[k + 2] : w[k];
#pragma unroll
    for (int k = 0; k < 5; ++k)
        w[k] = by1 ? w[k + 1] : w[k];
    Raw r;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        r.u[k] = DT != RED_F32 ? __funnelshift_r(w[k], w[k + 1], off << 3 & 16) : w[k];
    return r;
}
// Zeros from element n on.
template <int DT>
__device__ __forceinline__ Raw keep(Raw r, int n)
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (DT == RED_F32)
            r.u[k] = k < n ? r.u[k] : 0u;
        else
            r.u[k] = 2 * k + 1 < n ? r.u[k] : 2 * k < n ? r.u[k] & 0xffffu : 0u;
    }
    return r;
}

// A lane's units of a row (`row`: the row's first element); 0 behind its end.
// The loads are issued together: nothing here looks at what they bring.
template <int DT, bool VEC, int LANES, int N>
__device__ __forceinline__ void load_row(Raw (&r)[N], const void *p, int64_t row, int lane, int len)
{
    constexpr int E = UNIT<DT>, SIZE = 16 / E;
    const char *const at = static_cast<const char *>(p) + row * SIZE;
    if constexpr (VEC) {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int i = (u * LANES + lane) * E;
            const uint4 x = i + E <= len ? *reinterpret_cast<const uint4 *>(at + (int64_t)i * SIZE) : make_uint4(0, 0, 0, 0);
            r[u].u[0] = x.x, r[u].u[1] = x.y, r[u].u[2] = x.z, r[u].u[3] = x.w;
        }
        if (len % E == 0)
            return;
#pragma unroll
        for (int u = 0; u < N; ++u) {  // one lane's last unit
            const int i = (u * LANES + lane) * E;
            if (i < len && i + E > len)
                r[u] = load_some<DT>(p, row + i, len - i);
        }
    } else {
        const int off = block_offset(at);
        uint4 lo[N], hi[N];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int i = (u * LANES + lane) * E;
            const uint4 *const q = reinterpret_cast<const uint4 *>(at - off + (int64_t)i * SIZE);
            lo[u] = i < len ? q[0] : make_uint4(0, 0, 0, 0);
            hi[u] = i < len && (len - i) * SIZE + off > 16 ? q[1] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < N; ++u)
            r[u] = keep<DT>(window<DT>(lo[u], hi[u], off), len - (u * LANES + lane) * E);
    }
}

// Bytes lo .. hi of a block (whole elements), from `r`, which holds it in place.
template <int DT>
__device__ __forceinline__ void store_some(char *block, const Raw &r, int lo, int hi)
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (DT == RED_F32) {
            if (4 * k >= lo && 4 * k < hi)
                *reinterpret_cast<uint32_t *>(block + 4 * k) = r.u[k];
        } else {
            if (4 * k >= lo && 4 * k < hi)
                *reinterpret_cast<uint16_t *>(block + 4 * k) = (uint16_t)r.u[k];
            if (4 * k + 2 >= lo && 4 * k + 2 < hi)
                *reinterpret_cast<uint16_t *>(block + 4 * k + 2) = (uint16_t)(r.u[k] >> 16);
        }
    }
}

// Unit i / E of a row, of which the first len - i elements are written, where `here`.
// All lanes of the warp call it, with neighbouring units of a row in the lanes of a group.
template <int DT, bool VEC, int LANES>
__device__ __forceinline__ void store_unit(void *p, int64_t row, int i, int len, bool here, const float (&v)[UNIT<DT>])
{
    constexpr int E = UNIT<DT>, SIZE = 16 / E, W = LANES < 32 ? LANES : 32;
    const Raw r = narrow<DT>(v);
    char *const at = static_cast<char *>(p) + (row + i) * SIZE;
    if constexpr (VEC) {
        if (!here)
            return;
        if (i + E <= len)
            *reinterpret_cast<uint4 *>(at) = make_uint4(r.u[0], r.u[1], r.u[2], r.u[3]);
        else if (i < len)
            store_some<DT>(at, r, 0, (len - i) * SIZE);
    } else {
        const int off = block_offset(at);
        uint4 before;
        before.x = __shfl_up_sync(0xffffffffu, r.u[0], 1, W);
        before.y = __shfl_up_sync(0xffffffffu, r.u[1], 1, W);
        before.z = __shfl_up_sync(0xffffffffu, r.u[2], 1, W);
        before.w = __shfl_up_sync(0xffffffffu, r.u[3], 1, W);
        if (!here || i >= len)
            return;
        const int bytes = min(len - i, E) * SIZE, lane = threadIdx.x % W;
        const uint4 own = make_uint4(r.u[0], r.u[1], r.u[2], r.u[3]);
        // the block that this unit begins in: the end of the lane's before, and what fits of its own
        const Raw block = off == 0 ? r : window<DT>(before, own, 16 - off);
        const int lo = lane == 0 ? off : 0, hi = min(off + bytes, 16);
        if (lo == 0 && hi == 16)
            *reinterpret_cast<uint4 *>(at - off) = make_uint4(block.u[0], block.u[1], block.u[2], block.u[3]);
        else
            store_some<DT>(at - off, block, lo, hi);
        // the rest, where no lane behind takes it
        if (off + bytes > 16 && (lane == W - 1 || i + E >= len))
            store_some<DT>(at - off + 16, window<DT>(own, own, 16 - off), 0, off + bytes - 16);
    }
}

// ------------------------------------------------------- rows fetched ahead

template <bool KEEP>  // in L1, where another lane wants the same block
__device__ __forceinline__ void fetch16(void *dst, const void *src, uint32_t bytes)
{
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (KEEP)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fetch_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A ring of rows in shared memory, fetched while earlier rows are at work: each
// thread fetches its own units of up to MOST matrices (`arrays` of them in a call: what one
// does without leaves room for another CTA) and reads them back itself, so that no
// barrier is needed.  Of rows off the 16-byte blocks (VEC false) it fetches the
// two blocks that a unit lies in.
template <int DT, bool VEC, int LANES, int N, int MOST>
struct Ring {
    static constexpr int NT = GROUP_CTA<LANES>, E = UNIT<DT>, SIZE = 16 / E, BLOCKS = VEC ? 1 : 2;
    static constexpr int ARRAY = N * BLOCKS * NT * 16, STAGE = MOST * ARRAY;
    // one row at work, one on its way; more are no use (norm 30000 x 512 bf16 with four 18.4 us, with two 17.3)
    static constexpr int STAGES = 2 * STAGE <= 204800 ? 2 : 1;
    // the longest fp32 rows off the blocks do not fit: they are loaded where they are wanted
    static constexpr bool LATE = STAGE > 212992;
    static constexpr size_t bytes(int arrays) { return LATE ? 0 : (size_t)ARRAY * arrays * STAGES; }

    unsigned char *ring;
    int arrays;

    __device__ __forceinline__ uint4 *slot(int stage, int array, int u) const
    {
        return reinterpret_cast<uint4 *>(ring) + ((stage * arrays + array) * N + u) * BLOCKS * NT + threadIdx.x;
    }
    __device__ __forceinline__ void fetch(int stage, int array, const void *p, int64_t row, int lane, int len) const
    {
        if (LATE)
            return;
        const char *const at = static_cast<const char *>(p) + row * SIZE;
        const int off = VEC ? 0 : block_offset(at);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int i = (u * LANES + lane) * E;
            uint4 *const to = slot(stage, array, u);
            if constexpr (VEC) {
                const int left = (len - i) * SIZE;
                const uint32_t bytes = left <= 0 ? 0 : left < 16 ? left : 16;
                fetch16<false>(to, bytes ? at + (int64_t)i * SIZE : at, bytes);
            } else {
                const char *const block = at - off + (int64_t)i * SIZE;
                const bool one = i < len, two = one && (len - i) * SIZE + off > 16;
                fetch16<true>(to, one ? block : at - off, one ? 16 : 0);
                fetch16<true>(to + NT, two ? block + 16 : at - off, two ? 16 : 0);
            }
        }
    }
    // `row` and `len` as they were fetched; `lane`'s unit u.
    __device__ __forceinline__ Raw take(int stage, int array, int u, const void *p, int64_t row, int lane, int len) const
    {
        const uint4 *const from = slot(stage, array, u);
        if constexpr (LATE) {
            Raw r[1];
            load_row<DT, VEC, 1>(r, p, row + (u * LANES + lane) * E, 0, len - (u * LANES + lane) * E);
            return r[0];
        } else if constexpr (VEC) {
            const uint4 x = from[0];
            return {{x.x, x.y, x.z, x.w}};
        } else {
            const uint4 x = from[0];
            const int off = block_offset(static_cast<const char *>(p) + row * SIZE);
            return keep<DT>(window<DT>(x, from[NT], off), len - (u * LANES + lane) * E);
        }
    }
};

// ------------------------------------------------------------ group reduction

template <int LANES>
struct GroupShared {
    float2 part[2][LANES / 32];
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
            sh.part[turn][threadIdx.x / 32].x = v;
        __syncthreads();
        v = sh.part[turn][threadIdx.x % WARPS].x;
#pragma unroll
        for (int o = WARPS / 2; o; o >>= 1)
            v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
        turn ^= 1;
    }
    return v;
}

// Two sums at once: the second costs no latency of its own.
template <int LANES>
__device__ __forceinline__ float2 group_sums(float2 v, GroupShared<LANES> &sh, int &turn)
{
    auto add = [&](int o) {
        const float x = __shfl_xor_sync(0xffffffffu, v.x, o), y = __shfl_xor_sync(0xffffffffu, v.y, o);
        v.x += x;
        v.y += y;
    };
#pragma unroll
    for (int o = (LANES < 32 ? LANES : 32) / 2; o; o >>= 1)
        add(o);
    if constexpr (LANES > 32) {
        constexpr int WARPS = LANES / 32;
        if (threadIdx.x % 32 == 0)
            sh.part[turn][threadIdx.x / 32] = v;
        __syncthreads();
        v = sh.part[turn][threadIdx.x % WARPS];
#pragma unroll
        for (int o = WARPS / 2; o; o >>= 1)
            add(o);
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

// CTAs per SM of a kernel with one size of dynamic shared memory, per device.
struct Resident {
    std::atomic<int> per_sm[64] = {};
};

// CTAs of a persistent grid: what is resident at once, or what there is to do; at most `most`.
// `smem_most`: the most dynamic shared memory of any call of the kernel (its leave is the
// kernel's, not the call's).
template <class K>
int resident_grid(K kernel, Resident &cache, int threads, size_t smem, size_t smem_most, int64_t ctas, int64_t most,
                  unsigned *grid)
{
    DeviceInfo di;
    const int st = device_info(&di);
    if (st != RED_OK)
        return st;
    int per_sm = cache.per_sm[di.dev].load(std::memory_order_relaxed);
    if (per_sm == 0) {
        cudaError_t e = cudaSuccess;
        if (smem_most > 0)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_most);
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
