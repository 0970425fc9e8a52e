// red_rmsnorm.cuh -- root-mean-square norm of rows, with the residual's addition
// and an output in 8 bits with scales, and its backward:
//     t = x + residual,  rstd = 1 / sqrt(mean(t^2) + eps),  y = t * rstd * w;
//     h = t * rstd,  g = dy * w,  c = mean(g * h),
//     dx = rstd * (g - h * c) + dtotal,  dw = sum over rows of dy * h.
//
// Both directions are one pass: a group of lanes holds a row in registers, in
// fp32, between its reduction and its results, so that each matrix crosses
// memory once and that is what bounds them.  A group is 8 to 32 lanes of a warp
// (rows of up to 1024) or a CTA (up to 16384); a lane holds up to 32 elements.
// Rows are fetched into shared memory while earlier ones are at work (Ring in
// red_groups.cuh, and how rows off the 16-byte blocks of memory are read and written).
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
    int block, blocks;  // values of a block (a power of two below len) and blocks per row; 0 and 1: one scale per row
    int block_log2;
};
struct NormGradArgs {
    const void *dy, *x, *weight, *dtotal;
    const float *rstd;
    int64_t rows, ldy, ldx, ldt, ldd;
    int len;
    bool wide;
    float inv_len;
    void *dx, *dw;  // dw NULL: not wanted
    int wtype;      // of the weight and dw
    float *part;    // shares of dw, one of len per CTA
};

template <int DT>
int rmsnorm_forward(const NormArgs &a, int kind, cudaStream_t s);
template <int DT>
int rmsnorm_backward(const NormGradArgs &a, cudaStream_t s);

#ifdef RED_RMSNORM_DT  // the kernels of one direction (RED_RMSNORM_BACKWARD), for one type of x

namespace {

// A lane's weights, of x's type or fp32; 1 where there are none.  They are the same
// for every row of a group and stay in registers.  WIDE: fp32 beside rows of 16
// bits, whose units are two of the weight's.
template <int DT, bool WIDE, bool VEC, int LANES, int N>
struct Weights {
    static constexpr int E = UNIT<DT>, WT = WIDE ? RED_F32 : DT, WORDS = WIDE && DT != RED_F32 ? 8 : 4;
    uint32_t raw[N][WORDS];

    __device__ __forceinline__ Weights(const void *w, int lane, int len)
    {
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int h = 0; h < WORDS; h += 4) {
                constexpr int EW = UNIT<WT>;
                const int i = (u * LANES + lane) * E + h;
                Raw r;
                if (!w) {
                    float ones[EW];
#pragma unroll
                    for (int k = 0; k < EW; ++k)
                        ones[k] = 1.0f;
                    r = narrow<WT>(ones);
                } else if (VEC && i + EW <= len) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(static_cast<const char *>(w) + (int64_t)i * (16 / EW));
                    r = {{x.x, x.y, x.z, x.w}};
                } else {
                    r = load_some<WT>(w, i, len - i);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    raw[u][h + k] = r.u[k];
            }
    }
    __device__ __forceinline__ void at(int u, float (&w)[E]) const
    {
#pragma unroll
        for (int k = 0; k < E; ++k)
            w[k] = WT == RED_F32 ? __uint_as_float(raw[u][k % WORDS])
                                 : Elem<WT == RED_F32 ? RED_F16 : WT>::widen(raw[u][k / 2 % WORDS] >> (k % 2 * 16) & 0xffffu);
    }
};

#ifndef RED_RMSNORM_BACKWARD
// ----------------------------------------------------------------- forward

// The largest value of an 8-bit type.
template <int KIND>
constexpr float TOP = KIND == RED_QUANT_E4M3 ? 448.0f : 127.0f;

// The scale of values of at most `most` (a NaN stays one): not below 2^-126, where a scale has few digits
// and no inverse in fp32.  (Taking values and scale 2^64 times as large there costs 8 to 12% of every call: 16384 x
// 8192 f32 in e4m3 142 -> 160 us.)
template <int KIND>
__device__ __forceinline__ float scale_of(float most)
{
    return most == 0.0f ? 1.0f : Max()(most * (1.0f / TOP<KIND>), 1.175494351e-38f);
}

// A unit's values in 8 bits, to nearest, beyond the largest: the largest.  A product with
// the scale's inverse: it is off by 1.5 units of fp32's last place, which moves one
// value in a million across a border between two of 8 bits, and eight divisions
// cost more (16384 x 8192 bf16 178 us with them, 161 as it is; 4097 x 5120 42, 27).
template <int KIND, int E>
__device__ __forceinline__ uint64_t narrow8(const float (&v)[E], float inv)
{
    uint64_t r = 0;
#pragma unroll
    for (int k = 0; k < E; k += 2) {
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

// A unit's 8-bit values, as store_unit; off the blocks of E bytes (ALIGNED false) they
// are moved the same way.
template <int E, bool ALIGNED, int LANES>
__device__ __forceinline__ void store_q(uint8_t *q, int64_t row, int i, int len, bool here, uint64_t v)
{
    using Block = std::conditional_t<E == 8, uint64_t, uint32_t>;
    constexpr int W = LANES < 32 ? LANES : 32;
    uint8_t *const at = q + row + i;
    auto some = [](uint8_t *block, Block bits, int lo, int hi) {
#pragma unroll
        for (int k = 0; k < E; ++k)
            if (k >= lo && k < hi)
                block[k] = (uint8_t)(bits >> (8 * k));
    };
    const Block own = (Block)v;
    if constexpr (ALIGNED) {
        if (here && i + E <= len)
            *reinterpret_cast<Block *>(at) = own;
        else if (here && i < len)
            some(at, own, 0, len - i);
    } else {
        const int off = (int)((uintptr_t)at % E), lane = threadIdx.x % W;
        const Block before = __shfl_up_sync(0xffffffffu, own, 1, W);
        if (!here || i >= len)
            return;
        const int bytes = min(len - i, E);
        const Block block = off == 0 ? own : (Block)(own << (8 * off)) | (Block)(before >> (8 * (E - off)));
        const int lo = lane == 0 ? off : 0, hi = min(off + bytes, E);
        if (lo == 0 && hi == E)
            *reinterpret_cast<Block *>(at - off) = block;
        else
            some(at - off, block, lo, hi);
        if (off + bytes > E && (lane == W - 1 || i + E >= len))
            some(at - off + E, (Block)(own >> (8 * (E - off))), 0, off + bytes - E);
    }
}

// KIND: 0 for y in x's type, else the 8-bit type.  LONE: no residual.
// (Registers are left to the compiler, but for two cases.  One that it makes 70 of, and three CTAs per SM: with 64, and
// four, 16384 x 4096 bf16 91 -> 83 us.  One that it makes 92 to 128 of, and two, where only x is read and y written: with
// 80, and three, 16384 x 5120 bf16 without a residual 62.8 -> 57.2, x 6144 69.5 -> 63.2; but with one 106.0 -> 117.2
// (2000 rows 12.6 -> 11.8), in e4m3 with one 93.9 -> 98.5 and without 68.4 -> 72.5.  A bound of one CTA per SM has it
// take more than 128: 16384 x 8192 173 -> 264; 80 for rows that long are too few: 85 -> 104.)
template <int LANES, int VECS, bool VEC, bool RING, bool LONE>
constexpr int NORM_CTAS = LANES == 256 && VEC ? (VECS == 2 && !RING ? 4 : VECS == 3 && LONE ? 3 : 0) : 0;
template <int DT, bool WIDE, int KIND, int LANES, int VECS, bool VEC, bool RING, bool LONE>
__global__ void __launch_bounds__(GROUP_CTA<LANES>, NORM_CTAS<LANES, VECS, VEC, RING, LONE>)
    rmsnorm_kernel(const NormArgs a)
{
    pdl_enter();
    __shared__ GroupShared<LANES> sh;
    constexpr int NT = GROUP_CTA<LANES>, GROUPS = NT / LANES, N = UNITS<DT, VECS>, E = UNIT<DT>;
    using Rows = Ring<DT, VEC, LANES, UNITS<DT, VECS>, 2>;
    extern __shared__ __align__(16) unsigned char ring[];
    const Rows rows = {ring, a.residual ? 2 : 1};
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    const int64_t step = (int64_t)gridDim.x * GROUPS, first = (int64_t)blockIdx.x * GROUPS + group;
    int turn = 0, stage = 0;
    auto fetch = [&](int64_t r, int to) {
        if (r < a.rows) {
            rows.fetch(to, 0, a.x, r * a.ldx, lane, a.len);
            if (a.residual)
                rows.fetch(to, 1, a.residual, r * a.ldr, lane, a.len);
        }
        fetch_commit();
    };
    if constexpr (RING) {
#pragma unroll
        for (int k = 0; k < Rows::STAGES - 1; ++k)
            fetch(first + k * step, k);
    }
    const Weights<DT, WIDE, VEC, LANES, N> weights(a.weight, lane, a.len);
    // every group of a CTA takes part in the shuffles to the end
    for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < a.rows; r0 += step) {
        const bool here = r0 + group < a.rows;
        const int64_t r = here ? r0 + group : a.rows - 1;
        Raw raw[N], res[N];
        if constexpr (RING) {
            fetch(r0 + group + (Rows::STAGES - 1) * step, (stage + Rows::STAGES - 1) % Rows::STAGES);
            fetch_wait<Rows::STAGES - 1>();
#pragma unroll
            for (int v = 0; v < N; ++v) {
                raw[v] = rows.take(stage, 0, v, a.x, r * a.ldx, lane, a.len);
                if (a.residual)
                    res[v] = rows.take(stage, 1, v, a.residual, r * a.ldr, lane, a.len);
            }
            stage = (stage + 1) % Rows::STAGES;
        } else {
            load_row<DT, VEC, LANES>(raw, a.x, r * a.ldx, lane, a.len);
            if (a.residual)
                load_row<DT, VEC, LANES>(res, a.residual, r * a.ldr, lane, a.len);
        }
        float t[N][E];
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < N; ++v) {
            widen<DT>(raw[v], t[v]);
            if (a.residual) {
                float s[E];
                widen<DT>(res[v], s);
#pragma unroll
                for (int k = 0; k < E; ++k)
                    t[v][k] += s[k];
            }
#pragma unroll
            for (int k = 0; k < E; ++k)
                sum = fmaf(t[v][k], t[v][k], sum);
        }
        if (a.residual) {
#pragma unroll
            for (int v = 0; v < N; ++v)
                store_unit<DT, VEC, LANES>(a.total, r * a.ldt, (v * LANES + lane) * E, a.len, here, t[v]);
        }
        sum = group_fold<LANES>(sum, sh, turn, Add());
        const float rstd = __frsqrt_rn(fmaf(sum, a.inv_len, a.eps));
        if (a.rstd && lane == 0 && here)
            a.rstd[r] = rstd;
        float most[N];
#pragma unroll
        for (int v = 0; v < N; ++v) {
            float w[E];
            weights.at(v, w);
            most[v] = 0.0f;
#pragma unroll
            for (int k = 0; k < E; ++k) {
                t[v][k] = t[v][k] * rstd * w[k];
                if (KIND != 0)
                    most[v] = Max()(most[v], fabsf(t[v][k]));
            }
            if (KIND == 0)
                store_unit<DT, VEC, LANES>(a.y, r * a.ldy, (v * LANES + lane) * E, a.len, here, t[v]);
        }
        if constexpr (KIND != 0) {
            if (a.block) {
                // a block is 4 to 32 neighbouring lanes' units
                const int lanes = a.block / E;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
#pragma unroll
                    for (int v = 0; v < N; ++v)
                        if (o < lanes)  // (the same for all)
                            most[v] = Max()(most[v], __shfl_xor_sync(0xffffffffu, most[v], o));
            } else {
#pragma unroll
                for (int v = 1; v < N; ++v)
                    most[0] = Max()(most[0], most[v]);
                most[0] = group_fold<LANES>(most[0], sh, turn, Max());
            }
#pragma unroll
            for (int v = 0; v < N; ++v) {
                const int i = (v * LANES + lane) * E;
                const float scale = scale_of<KIND>(a.block ? most[v] : most[0]);
                const float inv = __frcp_rn(scale);
                if (here && i < a.len && (a.block ? (i & (a.block - 1)) == 0 : i == 0))
                    a.scales[r * a.blocks + (i >> a.block_log2)] = scale;
                store_q<E, VEC, LANES>(static_cast<uint8_t *>(a.y), r * a.ldy, i, a.len, here, narrow8<KIND>(t[v], inv));
            }
        }
    }
}

#else
// ---------------------------------------------------------------- backward

__device__ __forceinline__ void store_typed(int type, void *p, int64_t i, float v)
{
    if (type == RED_F32)
        store_elem<RED_F32>(p, i, v);
    else if (type == RED_F16)
        store_elem<RED_F16>(p, i, v);
    else
        store_elem<RED_BF16>(p, i, v);
}

// Column i of this CTA's share of dw; the only CTA's is dw itself.
__device__ __forceinline__ void write_share(const NormGradArgs &a, int i, float v)
{
    if (gridDim.x == 1)
        store_typed(a.wtype, a.dw, i, v);
    else
        a.part[(int64_t)blockIdx.x * a.len + i] = v;
}

// (128 registers where shared memory has room for two CTAs: with 132, and one CTA, 16384 x 8192 bf16 177 us, 161 so.)
template <int DT, bool WIDE, int LANES, int VECS, bool VEC>
__global__ void __launch_bounds__(GROUP_CTA<LANES>, LANES == 256 && VECS == 4 && VEC ? 2 : 0) rmsnorm_grad_kernel(const NormGradArgs a)
{
    pdl_enter();
    __shared__ GroupShared<LANES> sh;
    constexpr int NT = GROUP_CTA<LANES>, GROUPS = NT / LANES, N = UNITS<DT, VECS>, E = UNIT<DT>;
    // groups of one warp or less meet in shared memory before the workspace
    __shared__ float meet[GROUPS > 1 ? NT / 32 * N * LANES * E : 1];
    using Rows = Ring<DT, VEC, LANES, UNITS<DT, VECS>, 3>;
    extern __shared__ __align__(16) unsigned char ring[];
    const Rows rows = {ring, a.dtotal ? 3 : 2};
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    const int64_t step = (int64_t)gridDim.x * GROUPS, first = (int64_t)blockIdx.x * GROUPS + group;
    int turn = 0, stage = 0;
    auto fetch = [&](int64_t r, int to) {
        if (r < a.rows) {
            rows.fetch(to, 0, a.x, r * a.ldx, lane, a.len);
            rows.fetch(to, 1, a.dy, r * a.ldy, lane, a.len);
            if (a.dtotal)
                rows.fetch(to, 2, a.dtotal, r * a.ldt, lane, a.len);
        }
        fetch_commit();
    };
#pragma unroll
    for (int k = 0; k < Rows::STAGES - 1; ++k)
        fetch(first + k * step, k);
    const Weights<DT, WIDE, VEC, LANES, N> weights(a.weight, lane, a.len);
    float dw[N][E];
#pragma unroll
    for (int v = 0; v < N; ++v)
#pragma unroll
        for (int k = 0; k < E; ++k)
            dw[v][k] = 0.0f;
    float rstd_next = first < a.rows ? a.rstd[first] : 0.0f;
    for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < a.rows; r0 += step) {
        const bool here = r0 + group < a.rows;
        const int64_t r = here ? r0 + group : a.rows - 1;
        const float rstd = rstd_next;
        if (r0 + group + step < a.rows)
            rstd_next = a.rstd[r0 + group + step];
        fetch(r0 + group + (Rows::STAGES - 1) * step, (stage + Rows::STAGES - 1) % Rows::STAGES);
        fetch_wait<Rows::STAGES - 1>();
        auto take = [&](int array, int v, const void *p, int64_t ld, float (&to)[E]) {
            widen<DT>(rows.take(stage, array, v, p, r * ld, lane, a.len), to);
        };
        float c = 0.0f;
#pragma unroll
        for (int v = 0; v < N; ++v) {
            float h[E], g[E], w[E];
            take(0, v, a.x, a.ldx, h);
            take(1, v, a.dy, a.ldy, g);
            weights.at(v, w);
#pragma unroll
            for (int k = 0; k < E; ++k) {
                h[k] *= rstd;
                if (here)
                    dw[v][k] = fmaf(g[k], h[k], dw[v][k]);
                c = fmaf(g[k] * w[k], h[k], c);
            }
        }
        c = group_fold<LANES>(c, sh, turn, Add()) * a.inv_len;
        // h and g again from shared memory: registers hold the weights and dw
#pragma unroll
        for (int v = 0; v < N; ++v) {
            float h[E], g[E], w[E], d[E];
            take(0, v, a.x, a.ldx, h);
            take(1, v, a.dy, a.ldy, g);
            weights.at(v, w);
            if (a.dtotal)
                take(2, v, a.dtotal, a.ldt, d);
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float n = fmaf(-h[k] * rstd, c, g[k] * w[k]);
                d[k] = a.dtotal ? fmaf(n, rstd, d[k]) : n * rstd;
            }
            store_unit<DT, VEC, LANES>(a.dx, r * a.ldd, (v * LANES + lane) * E, a.len, here, d);
        }
        stage = (stage + 1) % Rows::STAGES;
    }
    if (!a.dw)
        return;
    if constexpr (GROUPS > 1) {
        // the groups of a warp by shuffles, the warps through shared memory
#pragma unroll
        for (int v = 0; v < N; ++v)
#pragma unroll
            for (int k = 0; k < E; ++k) {
#pragma unroll
                for (int o = LANES; o < 32; o <<= 1)
                    dw[v][k] += __shfl_xor_sync(0xffffffffu, dw[v][k], o);
                if (threadIdx.x % 32 < LANES)
                    meet[(threadIdx.x / 32 * N + v) * LANES * E + lane * E + k] = dw[v][k];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < a.len; i += NT) {
            float sum = meet[i];
#pragma unroll
            for (int w = 1; w < NT / 32; ++w)
                sum += meet[w * N * LANES * E + i];
            write_share(a, i, sum);
        }
    } else {
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const int i = (v * LANES + lane) * E;
            if (gridDim.x > 1 && a.len % 4 == 0 && i + E <= a.len) {
#pragma unroll
                for (int k = 0; k < E; k += 4)
                    *reinterpret_cast<float4 *>(a.part + (int64_t)blockIdx.x * a.len + i + k) =
                        make_float4(dw[v][k], dw[v][k + 1], dw[v][k + 2], dw[v][k + 3]);
            } else {
#pragma unroll
                for (int k = 0; k < E; ++k)
                    if (i + k < a.len)
                        write_share(a, i + k, dw[v][k]);
            }
        }
    }
}

// dw from the CTAs' shares: 32 columns by 32 lanes of shares, in a fixed order.
constexpr int JOIN_TURNS = 32;
__global__ void __launch_bounds__(32 * JOIN_TURNS) rmsnorm_join_kernel(const NormGradArgs a, int parts)
{
    pdl_enter();
    __shared__ float sums[JOIN_TURNS][33];
    const int lane = threadIdx.x % 32, turn = threadIdx.x / 32, col = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (col < a.len) {
#pragma unroll 8
        for (int p = turn; p < parts; p += JOIN_TURNS)
            s += a.part[(int64_t)p * a.len + col];
    }
    sums[turn][lane] = s;
    __syncthreads();
    s = sums[lane][turn];  // column `turn` of the 32, a share per lane
    for (int o = 16; o; o >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0 && blockIdx.x * 32 + turn < a.len)
        store_typed(a.wtype, a.dw, blockIdx.x * 32 + turn, s);
}

#endif

// ---------------------------------------------------------------- launches

#ifndef RED_RMSNORM_BACKWARD
template <int DT, bool WIDE, int KIND, int LANES, int VECS, bool VEC, bool RING, bool LONE = false>
int forward(const NormArgs &a, cudaStream_t s)
{
    static Resident caches[2];
    Resident &cache = caches[a.residual != nullptr];
    constexpr int NT = GROUP_CTA<LANES>, GROUPS = NT / LANES;
    using Rows = Ring<DT, VEC, LANES, UNITS<DT, VECS>, 2>;
    const size_t smem = RING ? Rows::bytes(a.residual ? 2 : 1) : 0;
    auto *const kernel = rmsnorm_kernel<DT, WIDE, KIND, LANES, VECS, VEC, RING, LONE>;
    unsigned grid;
    const int st = resident_grid(kernel, cache, NT, smem, RING ? Rows::bytes(2) : 0, (a.rows + GROUPS - 1) / GROUPS,
                                 INT32_MAX, &grid);
    if (st != RED_OK)
        return st;
    count_launches(1);
    return cuda_fail(launch_pdl_dynamic(kernel, dim3(grid), dim3(NT), smem, s, a), "rmsnorm");
}

}  // namespace

template <int DT, bool WIDE, bool VEC>
int forward_of(const NormArgs &a, int kind, cudaStream_t s)
{
    return with_group((a.len + 7) / 8, [&](auto lanes, auto vecs) {
        constexpr int L = decltype(lanes)::value, V = decltype(vecs)::value;
        // Rows fetched ahead or loaded where they are wanted, us at bf16: without a residual 16384 x
        // 4096 43 / 54, in 8 bits 16384 x 8192 161 / 167 and 4097 x 5120 27 / 39, with a residual 8192 x 2048 20 / 22, 4097 x
        // 5120 28 / 36 -- but with two matrices read and two of 16 bits written, and most of the
        // lanes' units in use, 16384 x 4096 94 / 83, 16384 x 8192 186 / 172, 65536 x 1024 91 / 83, 60000 x
        // 640 (five eighths of the units) 52 / 65.  fp32 is the same either way.
        constexpr bool DIRECT = VEC && V != 3 && L * V >= 128 && DT != RED_F32;
        if constexpr (DIRECT) {
            if (kind == 0 && a.residual && a.len > 6 * L * V)
                return forward<DT, WIDE, 0, L, V, VEC, false>(a, s);
        }
        if constexpr (VEC && V == 3 && L == 256 && DT != RED_F32) {
            if (kind == 0 && !a.residual)
                return forward<DT, WIDE, 0, L, V, VEC, true, true>(a, s);
        }
        return kind == 0                ? forward<DT, WIDE, 0, L, V, VEC, true>(a, s)
               : kind == RED_QUANT_E4M3 ? forward<DT, WIDE, RED_QUANT_E4M3, L, V, VEC, true>(a, s)
                                        : forward<DT, WIDE, RED_QUANT_I8, L, V, VEC, true>(a, s);
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
int backward(NormGradArgs a, cudaStream_t s)
{
    static Resident caches[2];
    Resident &cache = caches[a.dtotal != nullptr];
    constexpr int NT = GROUP_CTA<LANES>, GROUPS = NT / LANES;
    using Rows = Ring<DT, VEC, LANES, UNITS<DT, VECS>, 3>;
    const size_t smem = Rows::bytes(a.dtotal ? 3 : 2);
    unsigned grid;
    auto *const kernel = rmsnorm_grad_kernel<DT, WIDE, LANES, VECS, VEC>;
    int st = resident_grid(kernel, cache, NT, smem, Rows::bytes(3), (a.rows + GROUPS - 1) / GROUPS,
                           (int64_t)(WS_PART_ELEMS / (size_t)a.len), &grid);
    if (st != RED_OK)
        return st;
    const bool join = a.dw && grid > 1;
    if (join) {
        Workspace ws;
        st = get_workspace(&ws);
        if (st != RED_OK)
            return st;
        a.part = static_cast<float *>(ws.part);
    }
    st = cuda_fail(launch_pdl_dynamic(kernel, dim3(grid), dim3(NT), smem, s, a),
                   "rmsnorm_grad");
    if (st != RED_OK)
        return st;
    count_launches(1);
    if (!join)
        return RED_OK;
    count_launches(1);
    return cuda_fail(launch_pdl(rmsnorm_join_kernel, dim3((unsigned)((a.len + 31) / 32)), dim3(32 * JOIN_TURNS), s, a,
                                (int)grid),
                     "rmsnorm_join");
}

}  // namespace

template <int DT, bool WIDE, bool VEC>
int backward_of(const NormGradArgs &a, cudaStream_t s)
{
    return with_group((a.len + 7) / 8, [&](auto lanes, auto vecs) {
        return backward<DT, WIDE, decltype(lanes)::value, decltype(vecs)::value, VEC>(a, s);
    });
}

template <int DT>
int rmsnorm_backward(const NormGradArgs &a, cudaStream_t s)
{
    const int elem = DT == RED_F32 ? 4 : 2;
    const bool vec = aligned_rows(a.x, a.ldx, a.rows, elem) && aligned_rows(a.dy, a.ldy, a.rows, elem) &&
                     aligned_rows(a.dtotal, a.ldt, a.rows, elem) && aligned_rows(a.dx, a.ldd, a.rows, elem) &&
                     aligned_rows(a.weight, 0, 1, 1);
    if (DT != RED_F32 && a.wide)
        return vec ? backward_of<DT, true, true>(a, s) : backward_of<DT, true, false>(a, s);
    return vec ? backward_of<DT, DT == RED_F32, true>(a, s)
               : backward_of<DT, DT == RED_F32, false>(a, s);
}

template int rmsnorm_backward<RED_RMSNORM_DT>(const NormGradArgs &, cudaStream_t);

#endif
#endif

}  // namespace red
