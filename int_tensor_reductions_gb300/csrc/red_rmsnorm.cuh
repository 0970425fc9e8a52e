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
// same code with loads of one element.  Rows are fetched into shared memory while
// earlier ones are at work (Ring in red_groups.cuh).
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

#ifdef RED_RMSNORM_DT  // the kernels of one direction (RED_RMSNORM_BACKWARD), for one type of x

namespace {

// A lane's weights, of x's type or fp32; 1 where there are none.  They are the same
// for every row of a group and stay in registers.
template <int DT, bool WIDE, bool VEC, int LANES, int VECS>
struct Weights {
    static constexpr int WT = WIDE ? RED_F32 : DT;
    Raw<WT> raw[VECS];

    __device__ __forceinline__ Weights(const void *w, int lane, int len)
    {
        load_row<WT, VEC, LANES>(raw, w, 0, lane, w ? len : 0);
        if (!w) {
            float ones[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
#pragma unroll
            for (int v = 0; v < VECS; ++v)
                raw[v] = narrow<WT>(ones);
        }
    }
    __device__ __forceinline__ void at(int v, float (&w)[8]) const { widen<WT>(raw[v], w); }
};

#ifndef RED_RMSNORM_BACKWARD
// ----------------------------------------------------------------- forward

// The largest value of an 8-bit type.
template <int KIND>
constexpr float TOP = KIND == RED_QUANT_E4M3 ? 448.0f : 127.0f;

// The scale of values of at most `most`, and its inverse (finite where the scale
// has none in fp32).
template <int KIND>
__device__ __forceinline__ float scale_of(float most, float *inv)
{
    const float scale = most == 0.0f ? 1.0f : most * (1.0f / TOP<KIND>);
    *inv = fminf(__frcp_rn(scale), 3.402823466e38f);
    return scale;
}

// Eight 8-bit values, to nearest, beyond the largest: the largest.  A product with
// the scale's inverse: it is off by 1.5 units of fp32's last place, which moves one
// value in a million across a border between two of 8 bits, and eight divisions
// took more time than all else (16384 x 8192 bf16 295 us with them, DIVNOW without).
template <int KIND>
__device__ __forceinline__ uint64_t narrow8(const float (&v)[8], float inv)
{
    uint64_t r = 0;
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        const float a = v[k] * inv, b = v[k + 1] * inv;
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
template <int DT, bool WIDE, int KIND, int LANES, int VECS, bool VEC>
__global__ void __launch_bounds__(GROUP_CTA<LANES>) rmsnorm_kernel(const NormArgs a)
{
    pdl_enter();
    __shared__ GroupShared<LANES> sh;
    constexpr int NT = GROUP_CTA<LANES>, GROUPS = NT / LANES;
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    int turn = 0;
    const Weights<DT, WIDE, VEC, LANES, VECS> weights(a.weight, lane, a.len);
    // every group of a CTA takes part in the shuffles to the end
    for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < a.rows; r0 += (int64_t)gridDim.x * GROUPS) {
        const bool here = r0 + group < a.rows;
        const int64_t r = here ? r0 + group : a.rows - 1;
        Raw<DT> raw[VECS], res[VECS];
        load_row<DT, VEC, LANES>(raw, a.x, r * a.ldx, lane, a.len);
        if (a.residual)
            load_row<DT, VEC, LANES>(res, a.residual, r * a.ldr, lane, a.len);
        float t[VECS][8];
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            widen<DT>(raw[v], t[v]);
            if (a.residual) {
                float s[8];
                widen<DT>(res[v], s);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    t[v][k] += s[k];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sum = fmaf(t[v][k], t[v][k], sum);
        }
        if (a.residual && here) {
#pragma unroll
            for (int v = 0; v < VECS; ++v)
                store8<DT, VEC>(a.total, r * a.ldt, (v * LANES + lane) * 8, a.len, t[v]);
        }
        sum = group_fold<LANES>(sum, sh, turn, Add());
        const float rstd = __frsqrt_rn(fmaf(sum, a.inv_len, a.eps));
        if (a.rstd && lane == 0 && here)
            a.rstd[r] = rstd;
        float top = 0.0f;
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            const int i = (v * LANES + lane) * 8;
            float w[8];
            weights.at(v, w);
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
                float inv;
                const float scale = scale_of<KIND>(most, &inv);
                if (here && i < a.len) {
                    if (lane % lanes == 0)
                        a.scales[r * a.blocks + i / a.block] = scale;
                    store_q<KIND>(static_cast<uint8_t *>(a.y), r * a.ldy, i, a.len, VEC, narrow8<KIND>(t[v], inv));
                }
            } else {
                top = Max()(top, most);
            }
        }
        if (KIND != 0 && !a.block) {
            top = group_fold<LANES>(top, sh, turn, Max());
            float inv;
            const float scale = scale_of<KIND>(top, &inv);
            if (here) {
                if (lane == 0)
                    a.scales[r] = scale;
#pragma unroll
                for (int v = 0; v < VECS; ++v)
                    store_q<KIND>(static_cast<uint8_t *>(a.y), r * a.ldy, (v * LANES + lane) * 8, a.len, VEC,
                                  narrow8<KIND>(t[v], inv));
            }
        }
    }
}

#else
// ---------------------------------------------------------------- backward

template <int DT, bool WIDE, int LANES, int VECS, bool VEC>
__global__ void __launch_bounds__(GROUP_CTA<LANES>) rmsnorm_grad_kernel(const NormGradArgs a)
{
    pdl_enter();
    __shared__ GroupShared<LANES> sh;
    constexpr int NT = GROUP_CTA<LANES>, GROUPS = NT / LANES;
    // groups of one warp or less meet in shared memory before the workspace
    __shared__ float meet[GROUPS > 1 ? VECS * LANES * 8 : 1];
    using Rows = Ring<DT, LANES, VECS, 3>;
    extern __shared__ __align__(16) unsigned char ring[];
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    const int64_t step = (int64_t)gridDim.x * GROUPS, first = (int64_t)blockIdx.x * GROUPS + group;
    int turn = 0, stage = 0;
    auto fetch = [&](int64_t r, int to) {
        if (r < a.rows) {
            Rows::fetch(ring, to, 0, a.x, r * a.ldx, lane, a.len);
            Rows::fetch(ring, to, 1, a.dy, r * a.ldy, lane, a.len);
            if (a.dtotal)
                Rows::fetch(ring, to, 2, a.dtotal, r * a.ldt, lane, a.len);
        }
        fetch_commit();
    };
    if constexpr (VEC) {
#pragma unroll
        for (int k = 0; k < Rows::STAGES - 1; ++k)
            fetch(first + k * step, k);
    }
    const Weights<DT, WIDE, VEC, LANES, VECS> weights(a.weight, lane, a.len);
    float dw[VECS][8];
#pragma unroll
    for (int v = 0; v < VECS; ++v)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            dw[v][k] = 0.0f;
    float rstd_next = first < a.rows ? a.rstd[first] : 0.0f;
    for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < a.rows; r0 += step) {
        const bool here = r0 + group < a.rows;
        const int64_t r = here ? r0 + group : a.rows - 1;
        Raw<DT> x[VECS], dy[VECS], dt[VECS];
        const float rstd = rstd_next;
        if (r0 + group + step < a.rows)
            rstd_next = a.rstd[r0 + group + step];
        if constexpr (VEC) {
            fetch(r0 + group + (Rows::STAGES - 1) * step, (stage + Rows::STAGES - 1) % Rows::STAGES);
            fetch_wait<Rows::STAGES - 1>();
            Rows::take(x, ring, stage, 0);
            Rows::take(dy, ring, stage, 1);
        } else {
            load_row<DT, VEC, LANES>(x, a.x, r * a.ldx, lane, a.len);
            load_row<DT, VEC, LANES>(dy, a.dy, r * a.ldy, lane, a.len);
            if (a.dtotal)
                load_row<DT, VEC, LANES>(dt, a.dtotal, r * a.ldt, lane, a.len);
        }
        float c = 0.0f;
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            float h[8], g[8], w[8];
            widen<DT>(x[v], h);
            widen<DT>(dy[v], g);
            weights.at(v, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                h[k] *= rstd;
                if (here)
                    dw[v][k] = fmaf(g[k], h[k], dw[v][k]);
                c = fmaf(g[k] * w[k], h[k], c);
            }
        }
        c = group_fold<LANES>(c, sh, turn, Add()) * a.inv_len;
        if constexpr (VEC) {
            if (a.dtotal)
                Rows::take(dt, ring, stage, 2);
            stage = (stage + 1) % Rows::STAGES;
        }
        if (!here)
            continue;
        // h and g again, from what the loads brought: registers for them would be other rows' loads in flight
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            float h[8], g[8], w[8], d[8];
            widen<DT>(x[v], h);
            widen<DT>(dy[v], g);
            weights.at(v, w);
            if (a.dtotal)
                widen<DT>(dt[v], d);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float n = fmaf(-h[k] * rstd, c, g[k] * w[k]);
                d[k] = a.dtotal ? fmaf(n, rstd, d[k]) : n * rstd;
            }
            store8<DT, VEC>(a.dx, r * a.ldd, (v * LANES + lane) * 8, a.len, d);
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

#endif

// ---------------------------------------------------------------- launches

#ifndef RED_RMSNORM_BACKWARD
template <int DT, bool WIDE, int KIND, int LANES, int VECS, bool VEC>
int forward(const NormArgs &a, cudaStream_t s)
{
    static Resident cache;
    constexpr int NT = GROUP_CTA<LANES>, GROUPS = NT / LANES;
    unsigned grid;
    const int st = resident_grid(rmsnorm_kernel<DT, WIDE, KIND, LANES, VECS, VEC>, cache, NT, 0, (a.rows + GROUPS - 1) / GROUPS,
                           INT32_MAX, &grid);
    if (st != RED_OK)
        return st;
    count_launches(1);
    return cuda_fail(launch_pdl(rmsnorm_kernel<DT, WIDE, KIND, LANES, VECS, VEC>, dim3(grid), dim3(NT), s, a), "rmsnorm");
}

}  // namespace

template <int DT, bool WIDE, bool VEC>
int forward_of(const NormArgs &a, int kind, cudaStream_t s)
{
    return with_group((a.len + 7) / 8, [&](auto lanes, auto vecs) {
        constexpr int L = decltype(lanes)::value, V = decltype(vecs)::value;
        return kind == 0               ? forward<DT, WIDE, 0, L, V, VEC>(a, s)
               : kind == RED_QUANT_E4M3 ? forward<DT, WIDE, RED_QUANT_E4M3, L, V, VEC>(a, s)
                                        : forward<DT, WIDE, RED_QUANT_I8, L, V, VEC>(a, s);
    });
}

template <int DT>
int rmsnorm_forward(const NormArgs &a, int kind, cudaStream_t s)
{
    const int elem = DT == RED_F32 ? 4 : 2;
    const bool vec = aligned_rows(a.x, a.ldx, a.rows, elem) && aligned_rows(a.residual, a.ldr, a.rows, elem) &&
                     aligned_rows(a.total, a.ldt, a.rows, elem) && aligned_rows(a.weight, 0, 1, 1) &&
                     (kind ? (uintptr_t)a.y % 8 == 0 && (a.rows < 2 || a.ldy % 8 == 0)
                           : aligned_rows(a.y, a.ldy, a.rows, elem));
    if (DT != RED_F32 && a.wide)
        return vec ? forward_of<DT, true, true>(a, kind, s) : forward_of<DT, true, false>(a, kind, s);
    return vec ? forward_of<DT, DT == RED_F32, true>(a, kind, s) : forward_of<DT, DT == RED_F32, false>(a, kind, s);
}

template int rmsnorm_forward<RED_RMSNORM_DT>(const NormArgs &, int, cudaStream_t);

#else
template <int DT, bool WIDE, int LANES, int VECS, bool VEC>
int backward(NormGradArgs a, int wtype, void *dw, cudaStream_t s)
{
    static Resident cache;
    constexpr int NT = GROUP_CTA<LANES>, GROUPS = NT / LANES;
    constexpr size_t SMEM = VEC ? Ring<DT, LANES, VECS, 3>::BYTES : 0;
    unsigned grid;
    int st = resident_grid(rmsnorm_grad_kernel<DT, WIDE, LANES, VECS, VEC>, cache, NT, SMEM, (a.rows + GROUPS - 1) / GROUPS,
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
    st = cuda_fail(launch_pdl_dynamic(rmsnorm_grad_kernel<DT, WIDE, LANES, VECS, VEC>, dim3(grid), dim3(NT), SMEM, s, a), "rmsnorm_grad");
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

template <int DT, bool WIDE, bool VEC>
int backward_of(const NormGradArgs &a, int wtype, void *dw, cudaStream_t s)
{
    return with_group((a.len + 7) / 8, [&](auto lanes, auto vecs) {
        return backward<DT, WIDE, decltype(lanes)::value, decltype(vecs)::value, VEC>(a, wtype, dw, s);
    });
}

template <int DT>
int rmsnorm_backward(const NormGradArgs &a, int wtype, void *dw, cudaStream_t s)
{
    const int elem = DT == RED_F32 ? 4 : 2;
    const bool vec = aligned_rows(a.x, a.ldx, a.rows, elem) && aligned_rows(a.dy, a.ldy, a.rows, elem) &&
                     aligned_rows(a.dtotal, a.ldt, a.rows, elem) && aligned_rows(a.dx, a.ldd, a.rows, elem) &&
                     aligned_rows(a.weight, 0, 1, 1);
    if (DT != RED_F32 && a.wide)
        return vec ? backward_of<DT, true, true>(a, wtype, dw, s) : backward_of<DT, true, false>(a, wtype, dw, s);
    return vec ? backward_of<DT, DT == RED_F32, true>(a, wtype, dw, s)
               : backward_of<DT, DT == RED_F32, false>(a, wtype, dw, s);
}

template int rmsnorm_backward<RED_RMSNORM_DT>(const NormGradArgs &, int, void *, cudaStream_t);

#endif
#endif

}  // namespace red
