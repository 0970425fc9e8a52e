// red_rmsnorm.cuh -- root-mean-square norm of rows, with the residual's addition
// and an output in 8 bits with scales, and its backward:
//     t = x + residual,  rstd = 1 / sqrt(mean(t^2) + eps),  y = t * rstd * w;
//     h = t * rstd,  g = dy * w,  c = mean(g * h),
//     dx = rstd * (g - h * c) + dtotal,  dw = sum over rows of dy * h.
//
// Both directions are one pass: a group of lanes holds a row in registers, in
// fp32, between its reduction and its results, so that each matrix crosses
// memory once and that is what bounds them.  A group is 8 to 32 lanes of a warp
// (rows of up to 1024) or a CTA (up to 16384); a lane holds up to four vectors
// of eight consecutive elements.  Rows off the 16-byte boundaries go through the
// same code with loads of one element.
//
// The backward keeps each lane's share of dw in registers over all the rows of
// its group; the groups' shares go to the workspace and a second kernel adds them
// in a fixed order.
#pragma once

#include "red.h"
#include "red_internal.h"
#include "red_groups.cuh"
#include "red_prims.cuh"

namespace red {

// Types have been checked; `wide`: the weight is fp32.
struct NormArgs {
    const void *x, *residual, *weight;
    int64_t rows, ldx, ldr;
    int len;
    bool wide;
    float eps, inv_len;
    void *y, *total;
    int64_t ldy, ldt;
    float *rstd, *scales;
    int block, blocks;  // values and number of blocks per row; 0: one scale per row
};
struct NormGradArgs {
    const void *dy, *x, *weight, *dtotal;
    const float *rstd;
    int64_t rows, ldy, ldx, ldt, ldd;
    int len;
    bool wide;
    float inv_len;
    void *dx;
    float *part;  // shares of dw, one of len per CTA; NULL: not wanted
};

template <int DT>
int rmsnorm_forward(const NormArgs &a, int kind, cudaStream_t s);
template <int DT>
int rmsnorm_backward(const NormGradArgs &a, int wtype, void *dw, cudaStream_t s);

#ifdef RED_RMSNORM_DT  // the kernels, for one type of x

namespace {

// Eight weights, of x's type or fp32; 1 where there are none.
template <int DT, bool VEC>
__device__ __forceinline__ void load_weight(const void *w, bool wide, int i, int len, float (&v)[8])
{
    if (!w) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = 1.0f;
    } else if (DT == RED_F32 || wide) {
        load8<RED_F32, VEC>(w, 0, i, len, v);
    } else {
        load8<DT, VEC>(w, 0, i, len, v);
    }
}

// ----------------------------------------------------------------- forward

// The largest value of an 8-bit type.
template <int KIND>
constexpr float TOP = KIND == RED_QUANT_E4M3 ? 448.0f : 127.0f;

// Eight 8-bit values, to nearest, beyond the largest: the largest.
template <int KIND>
__device__ __forceinline__ uint64_t narrow8(const float (&v)[8], float scale)
{
    uint64_t r = 0;
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        const float a = __fdiv_rn(v[k], scale), b = __fdiv_rn(v[k + 1], scale);
        uint32_t two;
        if constexpr (KIND == RED_QUANT_E4M3) {
            uint16_t h;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(b), "f"(a));
            two = h;
        } else {
            int x, y;
            asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(x) : "f"(a));
            asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(y) : "f"(b));
            two = ((uint32_t)x & 0xffu) | ((uint32_t)y & 0xffu) << 8;
        }
        r |= (uint64_t)two << (8 * k);
    }
    return r;
}

template <int KIND>
__device__ __forceinline__ void store_q(uint8_t *q, int64_t row, int i, int len, bool vec, uint64_t v)
{
    if (vec && i + 8 <= len) {
        *reinterpret_cast<uint64_t *>(q + row + i) = v;
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (i + k < len)
            q[row + i + k] = (uint8_t)(v >> (8 * k));
}

// KIND: 0 for y in x's type, else the 8-bit type.
template <int DT, int KIND, int LANES, int VECS, bool VEC>
__global__ void __launch_bounds__(GROUP_CTA<LANES>) rmsnorm_kernel(const NormArgs a)
{
    pdl_enter();
    __shared__ GroupShared<LANES> sh;
    constexpr int NT = GROUP_CTA<LANES>, GROUPS = NT / LANES;
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    int turn = 0;
    // every group of a CTA takes part in the shuffles to the end
    for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < a.rows; r0 += (int64_t)gridDim.x * GROUPS) {
        const bool here = r0 + group < a.rows;
        const int64_t r = here ? r0 + group : a.rows - 1;
        float t[VECS][8];
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < VECS; ++v)
            load8<DT, VEC>(a.x, r * a.ldx, (v * LANES + lane) * 8, a.len, t[v]);
        if (a.residual) {
#pragma unroll
            for (int v = 0; v < VECS; ++v) {
                float s[8];
                const int i = (v * LANES + lane) * 8;
                load8<DT, VEC>(a.residual, r * a.ldr, i, a.len, s);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    t[v][k] += s[k];
                if (here)
                    store8<DT, VEC>(a.total, r * a.ldt, i, a.len, t[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < VECS; ++v)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sum = fmaf(t[v][k], t[v][k], sum);
        sum = group_fold<LANES>(sum, sh, turn, Add());
        const float rstd = __frsqrt_rn(fmaf(sum, a.inv_len, a.eps));
        if (a.rstd && lane == 0 && here)
            a.rstd[r] = rstd;
        float top = 0.0f;
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            const int i = (v * LANES + lane) * 8;
            float w[8];
            load_weight<DT, VEC>(a.weight, a.wide, i, a.len, w);
            float most = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                t[v][k] = t[v][k] * rstd * w[k];
                if (KIND != 0)
                    most = Max()(most, fabsf(t[v][k]));
            }
            if constexpr (KIND == 0) {
                if (here)
                    store8<DT, VEC>(a.y, r * a.ldy, i, a.len, t[v]);
            } else if (a.block) {
                // a block is 4, 8, 16 or 32 neighbouring lanes' vectors
                const int lanes = min(a.block / 8, LANES < 32 ? LANES : 32);
                for (int o = lanes / 2; o; o >>= 1)
                    most = Max()(most, __shfl_xor_sync(0xffffffffu, most, o));
                const float scale = most == 0.0f ? 1.0f : __fdiv_rn(most, TOP<KIND>);
                if (here && i < a.len) {
                    if (lane % lanes == 0)
                        a.scales[r * a.blocks + i / a.block] = scale;
                    store_q<KIND>(static_cast<uint8_t *>(a.y), r * a.ldy, i, a.len, VEC, narrow8<KIND>(t[v], scale));
                }
            } else {
                top = Max()(top, most);
            }
        }
        if (KIND != 0 && !a.block) {
            top = group_fold<LANES>(top, sh, turn, Max());
            const float scale = top == 0.0f ? 1.0f : __fdiv_rn(top, TOP<KIND>);
            if (here) {
                if (lane == 0)
                    a.scales[r] = scale;
#pragma unroll
                for (int v = 0; v < VECS; ++v)
                    store_q<KIND>(static_cast<uint8_t *>(a.y), r * a.ldy, (v * LANES + lane) * 8, a.len, VEC,
                                  narrow8<KIND>(t[v], scale));
            }
        }
    }
}

// ---------------------------------------------------------------- backward

template <int DT, int LANES, int VECS, bool VEC>
__global__ void __launch_bounds__(GROUP_CTA<LANES>) rmsnorm_grad_kernel(const NormGradArgs a)
{
    pdl_enter();
    __shared__ GroupShared<LANES> sh;
    constexpr int NT = GROUP_CTA<LANES>, GROUPS = NT / LANES;
    // groups of one warp or less meet in shared memory before the workspace
    __shared__ float meet[GROUPS > 1 ? VECS * LANES * 8 : 1];
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    int turn = 0;
    float dw[VECS][8];
#pragma unroll
    for (int v = 0; v < VECS; ++v)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            dw[v][k] = 0.0f;
    for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < a.rows; r0 += (int64_t)gridDim.x * GROUPS) {
        const bool here = r0 + group < a.rows;
        const int64_t r = here ? r0 + group : a.rows - 1;
        const float rstd = a.rstd[r];
        float h[VECS][8], g[VECS][8];
        float c = 0.0f;
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            load8<DT, VEC>(a.x, r * a.ldx, (v * LANES + lane) * 8, a.len, h[v]);
            load8<DT, VEC>(a.dy, r * a.ldy, (v * LANES + lane) * 8, a.len, g[v]);
        }
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            const int i = (v * LANES + lane) * 8;
            float w[8];
            load_weight<DT, VEC>(a.weight, a.wide, i, a.len, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                h[v][k] *= rstd;
                if (here)
                    dw[v][k] = fmaf(g[v][k], h[v][k], dw[v][k]);
                g[v][k] *= w[k];
                c = fmaf(g[v][k], h[v][k], c);
            }
        }
        c = group_fold<LANES>(c, sh, turn, Add()) * a.inv_len;
        if (!here)
            continue;
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            const int i = (v * LANES + lane) * 8;
            float d[8];
            if (a.dtotal) {
                load8<DT, VEC>(a.dtotal, r * a.ldt, i, a.len, d);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    d[k] = fmaf(fmaf(-h[v][k], c, g[v][k]), rstd, d[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    d[k] = fmaf(-h[v][k], c, g[v][k]) * rstd;
            }
            store8<DT, VEC>(a.dx, r * a.ldd, i, a.len, d);
        }
    }
    if (!a.part)
        return;
    if constexpr (GROUPS > 1) {
        for (int turn_of = 0; turn_of < GROUPS; ++turn_of) {
            if (group == turn_of) {
#pragma unroll
                for (int v = 0; v < VECS; ++v)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float *m = &meet[(v * 8 + k) * LANES + lane];
                        *m = turn_of == 0 ? dw[v][k] : *m + dw[v][k];
                    }
            }
            __syncthreads();
        }
#pragma unroll
        for (int v = 0; v < VECS; ++v)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                dw[v][k] = meet[(v * 8 + k) * LANES + lane];
        if (group != 0)
            return;
    }
#pragma unroll
    for (int v = 0; v < VECS; ++v)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = (v * LANES + lane) * 8 + k;
            if (i < a.len)
                a.part[(int64_t)blockIdx.x * a.len + i] = dw[v][k];
        }
}

// dw from the CTAs' shares: 32 columns by 8 lanes of shares, in a fixed order.
__global__ void __launch_bounds__(256) rmsnorm_join_kernel(const float *part, int parts, int len, int wtype, void *dw)
{
    pdl_enter();
    __shared__ float sums[8][33];
    const int col = blockIdx.x * 32 + threadIdx.x % 32, turn = threadIdx.x / 32;
    float s = 0.0f;
    if (col < len) {
#pragma unroll 4
        for (int p = turn; p < parts; p += 8)
            s += part[(int64_t)p * len + col];
    }
    sums[turn][threadIdx.x % 32] = s;
    __syncthreads();
    if (turn == 0 && col < len) {
#pragma unroll
        for (int k = 1; k < 8; ++k)
            s += sums[k][threadIdx.x % 32];
        if (wtype == RED_F32)
            store_elem<RED_F32>(dw, col, s);
        else if (wtype == RED_F16)
            store_elem<RED_F16>(dw, col, s);
        else
            store_elem<RED_BF16>(dw, col, s);
    }
}

// ---------------------------------------------------------------- launches

template <int DT, int KIND, int LANES, int VECS, bool VEC>
int forward(const NormArgs &a, cudaStream_t s)
{
    static std::atomic<int> cache{0};
    constexpr int NT = GROUP_CTA<LANES>, GROUPS = NT / LANES;
    unsigned grid;
    const int st = resident_grid(rmsnorm_kernel<DT, KIND, LANES, VECS, VEC>, cache, NT, (a.rows + GROUPS - 1) / GROUPS,
                           INT32_MAX, &grid);
    if (st != RED_OK)
        return st;
    count_launches(1);
    return cuda_fail(launch_pdl(rmsnorm_kernel<DT, KIND, LANES, VECS, VEC>, dim3(grid), dim3(NT), s, a), "rmsnorm");
}

template <int DT, int LANES, int VECS, bool VEC>
int backward(NormGradArgs a, int wtype, void *dw, cudaStream_t s)
{
    static std::atomic<int> cache{0};
    constexpr int NT = GROUP_CTA<LANES>, GROUPS = NT / LANES;
    unsigned grid;
    int st = resident_grid(rmsnorm_grad_kernel<DT, LANES, VECS, VEC>, cache, NT, (a.rows + GROUPS - 1) / GROUPS,
                     (int64_t)(WS_PART_ELEMS / (size_t)a.len), &grid);
    if (st != RED_OK)
        return st;
    if (dw) {
        Workspace ws;
        st = get_workspace(&ws);
        if (st != RED_OK)
            return st;
        a.part = static_cast<float *>(ws.part);
    }
    st = cuda_fail(launch_pdl(rmsnorm_grad_kernel<DT, LANES, VECS, VEC>, dim3(grid), dim3(NT), s, a), "rmsnorm_grad");
    if (st != RED_OK || !dw) {
        count_launches(1);
        return st;
    }
    count_launches(2);
    return cuda_fail(launch_pdl(rmsnorm_join_kernel, dim3((unsigned)((a.len + 31) / 32)), dim3(256), s, a.part, (int)grid,
                                a.len, wtype, dw),
                     "rmsnorm_join");
}

}  // namespace

template <int DT>
int rmsnorm_forward(const NormArgs &a, int kind, cudaStream_t s)
{
    const int elem = DT == RED_F32 ? 4 : 2;
    const bool vec = aligned_rows(a.x, a.ldx, a.rows, elem) && aligned_rows(a.residual, a.ldr, a.rows, elem) &&
                     aligned_rows(a.total, a.ldt, a.rows, elem) && aligned_rows(a.weight, 0, 1, 1) &&
                     (kind ? (uintptr_t)a.y % 8 == 0 && (a.rows < 2 || a.ldy % 8 == 0) : aligned_rows(a.y, a.ldy, a.rows, elem));
    return with_group((a.len + 7) / 8, [&](auto lanes, auto vecs) {
        constexpr int L = decltype(lanes)::value, V = decltype(vecs)::value;
        switch (kind) {
        case 0: return vec ? forward<DT, 0, L, V, true>(a, s) : forward<DT, 0, L, V, false>(a, s);
        case RED_QUANT_E4M3:
            return vec ? forward<DT, RED_QUANT_E4M3, L, V, true>(a, s) : forward<DT, RED_QUANT_E4M3, L, V, false>(a, s);
        default:
            return vec ? forward<DT, RED_QUANT_I8, L, V, true>(a, s) : forward<DT, RED_QUANT_I8, L, V, false>(a, s);
        }
    });
}

template <int DT>
int rmsnorm_backward(const NormGradArgs &a, int wtype, void *dw, cudaStream_t s)
{
    const int elem = DT == RED_F32 ? 4 : 2;
    const bool vec = aligned_rows(a.x, a.ldx, a.rows, elem) && aligned_rows(a.dy, a.ldy, a.rows, elem) &&
                     aligned_rows(a.dtotal, a.ldt, a.rows, elem) && aligned_rows(a.dx, a.ldd, a.rows, elem) &&
                     aligned_rows(a.weight, 0, 1, 1);
    return with_group((a.len + 7) / 8, [&](auto lanes, auto vecs) {
        constexpr int L = decltype(lanes)::value, V = decltype(vecs)::value;
        return vec ? backward<DT, L, V, true>(a, wtype, dw, s) : backward<DT, L, V, false>(a, wtype, dw, s);
    });
}

template int rmsnorm_forward<RED_RMSNORM_DT>(const NormArgs &, int, cudaStream_t);
template int rmsnorm_backward<RED_RMSNORM_DT>(const NormGradArgs &, int, void *, cudaStream_t);

#endif

}  // namespace red
