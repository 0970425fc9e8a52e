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

// Log-probabilities only.
struct LogprobArgs {
    const int64_t *target;
    float *logp, *lse;
};

struct PolicyArgs {
    const int64_t *target;
    const float *old_logp, *ref_logp, *adv, *weight;  // ref_logp, weight may be NULL
    float clip_low, clip_high, kl, gscale;
    float *loss, *logp, *stats;
};

struct PolicyTerms {
    float loss;   // before the weight
    float drift;  // the KL estimate e^d - d - 1
    float clipped;
    float dlogp;
};

// L = -min(r A, clip(r, 1 - low, 1 + high) A) + kl (e^d - d - 1) with
// r = e^(logp - old) and d = ref - logp; its derivative by logp.
__device__ __forceinline__ PolicyTerms policy_terms(float logp, float old, float ref, bool has_ref, float adv,
                                                    float low, float high, float kl)
{
    PolicyTerms t;
    const float ratio = expf(logp - old);
    const float bounded = fminf(fmaxf(ratio, 1.0f - low), 1.0f + high);
    // a ratio that overflowed times no advantage is no gain, not a NaN
    const float a = adv == 0.0f ? 0.0f : ratio * adv;
    const float b = bounded * adv;
    const bool clipped = a > b;
    t.clipped = clipped ? 1.0f : 0.0f;
    t.loss = -(clipped ? b : a);
    t.dlogp = clipped ? 0.0f : -a;
    t.drift = 0.0f;
    if (has_ref && kl != 0.0f) {
        const float d = ref == logp ? 0.0f : ref - logp;  // equal infinities do not drift
        t.drift = exp_excess(d);
        t.loss += kl * t.drift;
        t.dlogp -= kl * expm1f(d);
    }
    return t;
}

struct DistillArgs {
    int k, vdtype;
    const int64_t *ids;
    const void *vals;
    const float *lse;     // NULL: the teacher's values are renormalised over the row
    const float *weight;  // may be NULL
    float gscale;
    float *loss, *stats;
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
int launch_logprob_grad(int dtype, const LogitRows &a, const int64_t *target, const float *lse, const float *dlogp,
                        cudaStream_t s);
int launch_policy(int dtype, const LogitRows &a, const PolicyArgs &p, cudaStream_t s);
int launch_distill(int dtype, const LogitRows &a, const DistillArgs &p, cudaStream_t s);
int launch_preference(int dtype, const LogitRows &a, const PreferenceArgs &p, cudaStream_t s);

}  // namespace red
