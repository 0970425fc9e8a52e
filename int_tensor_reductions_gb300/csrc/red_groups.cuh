// red_groups.cuh -- rows held in the registers of a group of lanes: loads and
// stores of eight consecutive elements per lane, reductions over the group, and
// the group that a row's length asks for.  8 to 32 lanes of a warp, or a whole
// CTA, hold a row; vector v of lane l starts at element (v * LANES + l) * 8.
#pragma once

#include <cstdint>
#include <type_traits>

#include "red_internal.h"
#include "red_loss.cuh"

namespace red {

// ------------------------------------------------------------- row access

// Eight consecutive elements from i on; those at or behind len are 0.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void *p, int64_t row, int i, int len, float (&v)[8])
{
    if (VEC && i + 8 <= len) {
        if constexpr (DT == RED_F32) {
            const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + row + i);
            const float4 a = q[0], b = q[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + row + i);
            const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[2 * k] = Elem<DT>::widen(u[k] & 0xffffu);
                v[2 * k + 1] = Elem<DT>::widen(u[k] >> 16);
            }
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = i + k < len ? load_elem<DT>(p, row + i + k) : 0.0f;
}

template <int DT, bool VEC>
__device__ __forceinline__ void store8(void *p, int64_t row, int i, int len, const float (&v)[8])
{
    if (VEC && i + 8 <= len) {
        if constexpr (DT == RED_F32) {
            float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + row + i);
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                u[k] = (uint32_t)Elem<DT>::narrow(v[2 * k]) | (uint32_t)Elem<DT>::narrow(v[2 * k + 1]) << 16;
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + row + i) = make_uint4(u[0], u[1], u[2], u[3]);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (i + k < len)
            store_elem<DT>(p, row + i + k, v[k]);
}

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

// Threads of a CTA: one group, or several in 256.
template <int LANES>
constexpr int GROUP_CTA = LANES > 32 ? LANES : 256;

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
    if (vecs <= 512)
        return RED_GROUP(256, 2);
    if (vecs <= 1024)
        return RED_GROUP(256, 4);
    return RED_GROUP(512, 4);
#undef RED_GROUP
}

// Whether a matrix's rows start on 16-byte boundaries (NULL: there is none).
inline bool aligned_rows(const void *p, int64_t ld, int64_t rows, int elem)
{
    return !p || ((uintptr_t)p % 16 == 0 && (rows < 2 || ld * elem % 16 == 0));
}

// CTAs of a persistent grid: what is resident at once, or what there is to do.
template <class K>
int resident_grid(K kernel, std::atomic<int> &cache, int threads, int64_t ctas, int64_t most, unsigned *grid)
{
    DeviceInfo di;
    const int st = device_info(&di);
    if (st != RED_OK)
        return st;
    const int per_sm = cached_occupancy(cache, (const void *)kernel, threads);
    int64_t cap = (int64_t)(per_sm > 0 ? per_sm : 1) * di.sms;
    cap = cap < most ? cap : most;
    *grid = (unsigned)(ctas < cap ? ctas : cap);
    return RED_OK;
}

}  // namespace red
