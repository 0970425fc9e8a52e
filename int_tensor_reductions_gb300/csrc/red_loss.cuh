// red_loss.cuh -- building blocks of the losses over rows of logits
// (red_logprob, red_distill, red_policy, red_preference).
//
// Every loss is a function of the scaled logits z = scale * x of a row
// through its log-softmax.  A row is reduced to its maximum m (of the raw
// logits) and l = sum_j 2^((x_j - m) * s2), s2 = scale * log2(e), so that
//     logp_y = scale * (x_y - m) - ln l,   lse = scale * m + ln l,
//     p_j    = 2^((x_j - m) * s2) / l.
// The difference x_j - m is taken before the product: a product first could
// overflow for logits near the type's lowest value (an additive mask) and
// leave inf - inf, and the difference keeps the argument's error relative to
// the distance from the maximum.  Partial (m, l) pairs combine by rescaling
// to the larger maximum; where no logit is finite m = -inf and l = 0.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "red.h"
#include "red_types.cuh"

namespace red {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float NEG_INF = -__builtin_huge_valf();

// Rows of logits and of their gradient.
struct LogitRows {
    const void *x;
    int64_t rows, ld;
    void *dx;  // NULL: no gradient
    int64_t ldd;
    int len;
    float scale;
};

__device__ __forceinline__ float ex2(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

template <int DT>
__device__ __forceinline__ float load_elem(const void *p, int64_t i)
{
    using T = typename Elem<DT>::T;
    const T v = static_cast<const T *>(p)[i];
    if constexpr (DT == RED_F32)
        return v;
    else
        return Elem<DT>::widen((uint32_t)v);
}

template <int DT>
__device__ __forceinline__ void store_elem(void *p, int64_t i, float v)
{
    using T = typename Elem<DT>::T;
    static_cast<T *>(p)[i] = Elem<DT>::narrow(v);
}

// Element i of a float vector of run-time type (RED_F32, RED_F16 or RED_BF16).
__device__ __forceinline__ float load_any(int dtype, const void *p, int64_t i)
{
    return dtype == RED_F32 ? load_elem<RED_F32>(p, i)
                            : (dtype == RED_F16 ? load_elem<RED_F16>(p, i) : load_elem<RED_BF16>(p, i));
}

// ------------------------------------------------------ softmax statistics

struct SoftStat {
    float m, l;
};

// The reference point of exponentials under the maximum m: m itself, or 0
// where nothing is finite yet (so that -inf - m stays -inf and a NaN logit
// still reaches the sum).
__device__ __forceinline__ float ref_of(float m) { return m == NEG_INF ? 0.0f : m; }

__device__ __forceinline__ SoftStat soft_join(SoftStat a, SoftStat b, float s2)
{
    SoftStat r;
    r.m = fmaxf(a.m, b.m);
    const float m = ref_of(r.m);
    r.l = a.l * ex2((a.m - m) * s2) + b.l * ex2((b.m - m) * s2);
    return r;
}

__device__ __forceinline__ SoftStat soft_warp(SoftStat a, float s2)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        SoftStat b;
        b.m = __shfl_xor_sync(0xffffffffu, a.m, off);
        b.l = __shfl_xor_sync(0xffffffffu, a.l, off);
        a = soft_join(a, b, s2);
    }
    return a;
}

// ------------------------------------------------------------- the losses

__device__ __forceinline__ bool valid_id(int64_t y, int len) { return y >= 0 && y < len; }

// e^d - d - 1 without the cancellation of its terms near zero: the series
// d^2/2 (1 + d/3 (1 + d/4 (1 + ...))) up to d^8/8! for |d| < 1/4 (the next
// term is below 2^-24 of the sum there).
__device__ __forceinline__ float exp_excess(float d)
{
    if (fabsf(d) < 0.25f) {
        float s = 1.0f + d * (1.0f / 8.0f);
        s = 1.0f + d * (1.0f / 7.0f) * s;
        s = 1.0f + d * (1.0f / 6.0f) * s;
        s = 1.0f + d * (1.0f / 5.0f) * s;
        s = 1.0f + d * (1.0f / 4.0f) * s;
        s = 1.0f + d * (1.0f / 3.0f) * s;
        return 0.5f * d * d * s;
    }
    return expf(d) - d - 1.0f;
}

enum : int { ROW_END = 0, ROW_OUT = 1, ROW_LIVE = 2 };

// What a kernel knows of a row before its logits: its index, whether it takes
// part, and the loss's inputs.
struct RowEntry {
    int64_t r;
    int64_t target;
    int state;    // ROW_*
    uint32_t xy;  // the target's logit, as stored
    float w;      // weight, or the gradient by logp
    float f[3];
};

// Element i of a row as stored, for load latency to pass before it is widened.
template <int DT>
__device__ __forceinline__ uint32_t load_bits(const void *p, int64_t i)
{
    if constexpr (DT == RED_F32)
        return static_cast<const uint32_t *>(p)[i];
    else
        return static_cast<const uint16_t *>(p)[i];
}

// The gradient of a row: g_j = mul * 2^(fma(x_j, fa, fb) * fc) + [j == y] cy,
// or zeros throughout.
struct RowGrad {
    float fa, fb, fc, mul, cy;
    int y;
    bool zero;
};

__device__ __forceinline__ bool row_empty(SoftStat t) { return t.m == NEG_INF && t.l == 0.0f; }

// c * ([j == y] - p_j) from the row's statistics.
__device__ __forceinline__ RowGrad grad_of_target(const LogitRows &a, SoftStat t, int y, float c)
{
    return RowGrad{1.0f, -t.m, a.scale * LOG2E, -c / t.l, c, y, row_empty(t) || c == 0.0f};
}

// Each loss below gives the kernels
//   STATS    whether a row's statistics come from its logits;
//   TEACHER  whether it has a list of teacher entries per row;
//   GRADIENT whether it can have a gradient;
//   load()   the row's entry (its logits are still intact): issues loads and
//            uses none of their values, so that a later settle() may be the
//            first to wait for them;
//   settle() whether the row takes part, and the load of the target's logit;
//   grad()   the row's gradient from entry and statistics (any thread);
//   write()  the row's scalar results (one thread), for rows out of the loss
//            too.

struct LogprobArgs {
    static constexpr bool STATS = true, TEACHER = false, GRADIENT = false;
    const int64_t *target;
    float *logp, *lse;

    __device__ void load(int64_t r, RowEntry &e) const
    {
        e.r = r;
        e.target = target[r];
    }
    template <int DT>
    __device__ void settle(const LogitRows &a, RowEntry &e) const
    {
        e.state = valid_id(e.target, a.len) ? ROW_LIVE : ROW_OUT;
        if (e.state == ROW_LIVE)
            e.xy = load_bits<DT>(a.x, e.r * a.ld + e.target);
    }
    template <int DT>
    __device__ RowGrad grad(const LogitRows &, const RowEntry &, SoftStat, float) const { return RowGrad{}; }
    template <int DT>
    __device__ void write(const LogitRows &a, const RowEntry &e, SoftStat t) const
    {
        float p = 0.0f, n = 0.0f;
        if (e.state == ROW_LIVE) {
            const float ln = logf(t.l);
            n = row_empty(t) ? NEG_INF : fmaf(a.scale, t.m, ln);
            p = row_empty(t) ? NEG_INF : (Elem<DT>::widen(e.xy) - t.m) * a.scale - ln;
        }
        logp[e.r] = p;
        lse[e.r] = n;
    }
};

struct LogprobGradArgs {
    static constexpr bool STATS = false, TEACHER = false, GRADIENT = true;
    const int64_t *target;
    const float *lse, *dlogp;

    __device__ void load(int64_t r, RowEntry &e) const
    {
        e.r = r;
        e.target = target[r];
        e.w = dlogp[r];
        e.f[0] = lse[r];
    }
    template <int DT>
    __device__ void settle(const LogitRows &a, RowEntry &e) const
    {
        e.state = valid_id(e.target, a.len) && e.w != 0.0f && e.f[0] != NEG_INF ? ROW_LIVE : ROW_OUT;
    }
    // p_j = 2^((scale x_j - lse) log2 e): the difference in one rounding, so
    // that it is exact where p_j is near 1.
    template <int DT>
    __device__ RowGrad grad(const LogitRows &a, const RowEntry &e, SoftStat, float) const
    {
        const float c = e.w * a.scale;
        return RowGrad{a.scale, -e.f[0], LOG2E, -c, c, (int)e.target, false};
    }
    template <int DT>
    __device__ void write(const LogitRows &, const RowEntry &, SoftStat) const {}
};

struct PolicyTerms {
    float loss;   // before the weight
    float drift;  // the KL estimate e^d - d - 1
    float clipped;
    float dlogp;
};

struct PolicyArgs {
    static constexpr bool STATS = true, TEACHER = false, GRADIENT = true;
    const int64_t *target;
    const float *old_logp, *ref_logp, *adv, *weight;  // ref_logp, weight may be NULL
    float clip_low, clip_high, kl, gscale;
    float *loss, *logp, *stats;

    // L = -min(r A, clip(r, 1 - low, 1 + high) A) + kl (e^d - d - 1) with
    // r = e^(logp - old) and d = ref - logp; its derivative by logp.
    __device__ PolicyTerms terms(float lp, float old, float ref, float A) const
    {
        PolicyTerms t;
        const float ratio = expf(lp - old);
        const float bounded = fminf(fmaxf(ratio, 1.0f - clip_low), 1.0f + clip_high);
        // a ratio that overflowed times no advantage is no gain, not a NaN
        const float free = A == 0.0f ? 0.0f : ratio * A;
        const float held = bounded * A;
        const bool clipped = free > held;
        t.clipped = clipped ? 1.0f : 0.0f;
        t.loss = -(clipped ? held : free);
        t.dlogp = clipped ? 0.0f : -free;
        t.drift = 0.0f;
        if (ref_logp && kl != 0.0f) {
            const float d = ref == lp ? 0.0f : ref - lp;  // equal infinities do not drift
            t.drift = exp_excess(d);
            t.loss += kl * t.drift;
            t.dlogp -= kl * expm1f(d);
        }
        return t;
    }
    __device__ void load(int64_t r, RowEntry &e) const
    {
        e.r = r;
        e.target = target[r];
        e.w = weight ? weight[r] : 1.0f;
        e.f[0] = old_logp[r];
        e.f[1] = ref_logp ? ref_logp[r] : 0.0f;
        e.f[2] = adv[r];
    }
    template <int DT>
    __device__ void settle(const LogitRows &a, RowEntry &e) const
    {
        e.state = valid_id(e.target, a.len) && e.w != 0.0f ? ROW_LIVE : ROW_OUT;
        if (e.state == ROW_LIVE)
            e.xy = load_bits<DT>(a.x, e.r * a.ld + e.target);
    }
    template <int DT>
    __device__ float row_logp(const LogitRows &a, const RowEntry &e, SoftStat t) const
    {
        return (Elem<DT>::widen(e.xy) - t.m) * a.scale - logf(t.l);
    }
    template <int DT>
    __device__ RowGrad grad(const LogitRows &a, const RowEntry &e, SoftStat t, float) const
    {
        const PolicyTerms q = terms(row_logp<DT>(a, e, t), e.f[0], e.f[1], e.f[2]);
        return grad_of_target(a, t, (int)e.target, e.w * q.dlogp * gscale * a.scale);
    }
    template <int DT>
    __device__ void write(const LogitRows &a, const RowEntry &e, SoftStat t) const
    {
        float p = 0.0f, v = 0.0f;
        if (e.state == ROW_LIVE && row_empty(t)) {
            p = NEG_INF;
        } else if (e.state == ROW_LIVE) {
            p = row_logp<DT>(a, e, t);
            v = e.w * terms(p, e.f[0], e.f[1], e.f[2]).loss;
        }
        logp[e.r] = p;
        loss[e.r] = v;
    }
};

// Teacher entries of a row in shared memory, k of each.
struct TeacherRow {
    int *id;    // column, -1: no entry, or merged into an earlier one
    float *q;   // probability
    float *lq;  // its logarithm
    float *x;   // the student's logit
};

struct DistillArgs {
    static constexpr bool STATS = true, TEACHER = true, GRADIENT = true;
    int k, vdtype;
    const int64_t *ids;
    const void *vals;
    const float *lse;     // NULL: the teacher's values are renormalised over the row
    const float *weight;  // may be NULL
    float gscale;
    float *loss, *stats;

    __device__ void load(int64_t r, RowEntry &e) const
    {
        e.r = r;
        e.w = weight ? weight[r] : 1.0f;
    }
    template <int DT>
    __device__ void settle(const LogitRows &, RowEntry &e) const
    {
        e.state = e.w != 0.0f ? ROW_LIVE : ROW_OUT;
    }
    template <int DT>
    __device__ RowGrad grad(const LogitRows &a, const RowEntry &e, SoftStat t, float Q) const
    {
        const float s2 = a.scale * LOG2E, c = e.w * gscale * a.scale;
        return RowGrad{1.0f, -t.m, s2, c * Q / t.l, 0.0f, -1, row_empty(t)};
    }
    template <int DT>
    __device__ void write(const LogitRows &, const RowEntry &, SoftStat) const {}

    // Teacher probabilities of a row, by a whole warp; returns Q = sum q.
    template <int DT>
    __device__ float prepare(const LogitRows &a, int64_t r, TeacherRow s) const
    {
        const int lane = threadIdx.x & 31;
        float vmax = NEG_INF;
        for (int i = lane; i < k; i += 32) {
            const int64_t id = ids[r * k + i];
            const bool ok = valid_id(id, a.len);
            const float v = ok ? load_any(vdtype, vals, r * k + i) * a.scale : NEG_INF;
            s.id[i] = ok ? (int)id : -1;
            s.lq[i] = v;
            s.x[i] = ok ? load_elem<DT>(a.x, r * a.ld + id) : 0.0f;
            vmax = fmaxf(vmax, v);
        }
        float norm;
        if (lse) {
            norm = lse[r];
        } else {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, off));
            float sum = 0.0f;
            for (int i = lane; i < k; i += 32)
                sum += expf(s.lq[i] - ref_of(vmax));
            sum = warp_sum(sum);
            norm = vmax == NEG_INF && sum == 0.0f ? 0.0f : vmax + logf(sum);
        }
        float Q = 0.0f;
        for (int i = lane; i < k; i += 32) {
            const float lq = s.lq[i] - norm;
            const float q = s.id[i] < 0 ? 0.0f : expf(lq);
            s.lq[i] = lq;
            s.q[i] = q;
            Q += q;
        }
        __syncwarp();
        return warp_sum(Q);
    }
    // The row's loss, by a whole warp; `t` holds the student's statistics.
    __device__ void finish(const LogitRows &a, const RowEntry &e, SoftStat t, TeacherRow s) const
    {
        const int lane = threadIdx.x & 31;
        float v = 0.0f;
        if (e.state == ROW_LIVE && !row_empty(t)) {
            const float ln = logf(t.l);
            for (int i = lane; i < k; i += 32)
                if (s.q[i] != 0.0f)
                    v += s.q[i] * (s.lq[i] - ((s.x[i] - t.m) * a.scale - ln));
            v = warp_sum(v) * e.w;
        }
        if (lane == 0)
            loss[e.r] = v;
    }
    // The teacher's columns of the gradient once more, by a whole warp after
    // the rest of the row is written: g_id = mul 2^(...) - c q.  An id that
    // comes more than once is written by its first entry.
    template <int DT>
    __device__ void patch(const LogitRows &a, const RowEntry &e, RowGrad g, TeacherRow s) const
    {
        const float c = e.w * gscale * a.scale;
        for (int i = threadIdx.x & 31; i < k; i += 32) {
            const int id = s.id[i];
            if (id < 0)
                continue;
            float q = 0.0f;
            bool first = true;
            for (int j = 0; j < k; ++j)
                if (s.id[j] == id) {
                    first = first && j >= i;
                    q += s.q[j];
                }
            if (first)
                store_elem<DT>(a.dx, e.r * a.ldd + id, g.mul * ex2(fmaf(s.x[i], g.fa, g.fb) * g.fc) - c * q);
        }
    }
    static __device__ __forceinline__ float warp_sum(float v)
    {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, off);
        return v;
    }
};

struct PreferenceArgs {
    int64_t pairs;
    const int64_t *target, *offsets;
    const float *ref_logp, *weight;  // may be NULL
    int kind, average;
    float beta, margin, smoothing, gscale;
    float *loss, *seq_logp, *stats;
    float *logp, *lse, *dlogp, *u;  // scratch of the caller: rows, rows, rows and pairs floats
};

// Launchers: arguments have been validated by the entry points.
int launch_logprob(int dtype, const LogitRows &a, const LogprobArgs &p, cudaStream_t s);
int launch_logprob_grad(int dtype, const LogitRows &a, const LogprobGradArgs &p, cudaStream_t s);
int launch_policy(int dtype, const LogitRows &a, const PolicyArgs &p, cudaStream_t s);
int launch_distill(int dtype, const LogitRows &a, const DistillArgs &p, cudaStream_t s);
int launch_preference(int dtype, const LogitRows &a, const PreferenceArgs &p, cudaStream_t s);

}  // namespace red
