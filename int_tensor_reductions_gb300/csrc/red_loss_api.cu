// red_loss_api.cu -- the extern "C" entry points of the losses over rows of
// logits (declared and documented in red.h): argument checks before any
// launch.
#include <cmath>

#include "red_internal.h"
#include "red_loss.cuh"

using namespace red;

namespace {

constexpr int64_t MAX_ELEMS = int64_t(1) << 44;
constexpr int64_t MAX_LEN = int64_t(1) << 30;  // row positions are 32-bit in the kernels

bool bad_ptr(const void *p, uintptr_t align) { return !p || ((uintptr_t)p) % align != 0; }
bool bad_opt(const void *p, uintptr_t align) { return p && ((uintptr_t)p) % align != 0; }
uintptr_t elem_size(int dtype) { return dtype == RED_F32 ? 4 : 2; }
bool float_type(int dtype) { return dtype == RED_F32 || dtype == RED_F16 || dtype == RED_BF16; }

// The checks every loss shares; RED_OK with `a` filled in.
int logit_rows(const char *who, int dtype, const void *x, int64_t rows, int64_t len, int64_t ld, float scale,
               void *dx, int64_t ldd, bool need_dx, LogitRows *a)
{
    if (!float_type(dtype))
        return fail(RED_EINVAL, "%s: dtype %d is not RED_F32, RED_F16 or RED_BF16", who, dtype);
    if (rows < 0 || rows > MAX_ELEMS || len < 1 || len > MAX_LEN)
        return fail(RED_EINVAL, "%s: rows = %lld, len = %lld out of range", who, (long long)rows, (long long)len);
    if (ld < len || ld > MAX_ELEMS || (rows > 0 && ld > MAX_ELEMS / rows))
        return fail(RED_EINVAL, "%s: row stride ld = %lld must be >= len = %lld and rows * ld in range", who,
                    (long long)ld, (long long)len);
    if (!(scale >= 1e-30f && scale <= 1e30f))
        return fail(RED_EINVAL, "%s: scale must be in 1e-30..1e30", who);
    if (dx || need_dx) {
        if (ldd < len || ldd > MAX_ELEMS || (rows > 0 && ldd > MAX_ELEMS / rows))
            return fail(RED_EINVAL, "%s: gradient row stride ldd = %lld must be >= len = %lld and rows * ldd in range",
                        who, (long long)ldd, (long long)len);
        if (dx == x && ldd != ld && rows > 1)
            return fail(RED_EINVAL, "%s: a gradient in place of the logits needs ldd == ld", who);
    }
    if (rows > 0) {
        if (bad_ptr(x, elem_size(dtype)))
            return fail(RED_EINVAL, "%s: x is NULL or not aligned to its element size", who);
        if (need_dx ? bad_ptr(dx, elem_size(dtype)) : bad_opt(dx, elem_size(dtype)))
            return fail(RED_EINVAL, "%s: dx is NULL or not aligned to its element size", who);
    }
    const double log2e = 1.4426950408889634074;
    const float s2 = (float)(scale * log2e);
    const double ratio = (double)s2 / scale;
    *a = LogitRows{x, rows, ld, dx, ldd, (int)len, scale, s2, (float)ratio, (float)(ratio - (double)(float)ratio)};
    return RED_OK;
}

int zero_stats(const char *who, float *stats, int n, cudaStream_t s)
{
    return cuda_fail(cudaMemsetAsync(stats, 0, n * sizeof(float), s), who);
}

}  // namespace

extern "C" {

int red_logprob(int dtype, const void *x, int64_t rows, int64_t len, int64_t ld, float scale, const int64_t *target,
                float *logp, float *lse, red_stream_t stream)
{
    LogitRows a;
    const int st = logit_rows("red_logprob", dtype, x, rows, len, ld, scale, nullptr, 0, false, &a);
    if (st != RED_OK)
        return st;
    if (rows == 0)
        return RED_OK;
    if (bad_ptr(target, 8))
        return fail(RED_EINVAL, "red_logprob: target is NULL or not 8-byte aligned");
    if (bad_ptr(logp, 4) || bad_ptr(lse, 4))
        return fail(RED_EINVAL, "red_logprob: logp or lse is NULL or not 4-byte aligned");
    return launch_logprob(dtype, a, LogprobArgs{target, logp, lse, nullptr, 0}, reinterpret_cast<cudaStream_t>(stream));
}

int red_logprob_grad(int dtype, const void *x, int64_t rows, int64_t len, int64_t ld, float scale,
                     const int64_t *target, const float *lse, const float *dlogp, void *dx, int64_t ldd,
                     red_stream_t stream)
{
    LogitRows a;
    const int st = logit_rows("red_logprob_grad", dtype, x, rows, len, ld, scale, dx, ldd, true, &a);
    if (st != RED_OK)
        return st;
    if (rows == 0)
        return RED_OK;
    if (bad_ptr(target, 8))
        return fail(RED_EINVAL, "red_logprob_grad: target is NULL or not 8-byte aligned");
    if (bad_ptr(lse, 4) || bad_ptr(dlogp, 4))
        return fail(RED_EINVAL, "red_logprob_grad: lse or dlogp is NULL or not 4-byte aligned");
    return launch_logprob_grad(dtype, a, LogprobGradArgs{target, lse, dlogp, nullptr, rows}, reinterpret_cast<cudaStream_t>(stream));
}

int red_distill(int dtype, const void *x, int64_t rows, int64_t len, int64_t ld, float scale, int64_t k,
                const int64_t *ids, int vdtype, const void *vals, const float *lse, const float *weight,
                float grad_scale, float *loss, float *stats, void *dx, int64_t ldd, red_stream_t stream)
{
    LogitRows a;
    const int st = logit_rows("red_distill", dtype, x, rows, len, ld, scale, dx, ldd, false, &a);
    if (st != RED_OK)
        return st;
    if (k < 1 || k > RED_DISTILL_MAX_K)
        return fail(RED_EINVAL, "red_distill: k = %lld outside 1..%d", (long long)k, RED_DISTILL_MAX_K);
    if (!float_type(vdtype))
        return fail(RED_EINVAL, "red_distill: vdtype %d is not RED_F32, RED_F16 or RED_BF16", vdtype);
    if (std::isnan(grad_scale) || std::isinf(grad_scale))
        return fail(RED_EINVAL, "red_distill: grad_scale must be finite");
    if (bad_ptr(stats, 4))
        return fail(RED_EINVAL, "red_distill: stats is NULL or not 4-byte aligned");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0)
        return zero_stats("red_distill: cudaMemsetAsync", stats, 2, s);
    if (bad_ptr(ids, 8) || bad_ptr(vals, elem_size(vdtype)))
        return fail(RED_EINVAL, "red_distill: ids or vals is NULL or not aligned to its element size");
    if (bad_opt(lse, 4) || bad_opt(weight, 4) || bad_ptr(loss, 4))
        return fail(RED_EINVAL, "red_distill: loss is NULL, or lse, weight or loss is not 4-byte aligned");
    return launch_distill(dtype, a, DistillArgs{(int)k, vdtype, ids, vals, lse, weight, grad_scale, loss, stats}, s);
}

int red_policy(int dtype, const void *x, int64_t rows, int64_t len, int64_t ld, float scale, const int64_t *target,
               const float *old_logp, const float *ref_logp, const float *adv, const float *weight, float clip_low,
               float clip_high, float kl_coef, float grad_scale, float *loss, float *logp, float *stats, void *dx,
               int64_t ldd, red_stream_t stream)
{
    LogitRows a;
    const int st = logit_rows("red_policy", dtype, x, rows, len, ld, scale, dx, ldd, false, &a);
    if (st != RED_OK)
        return st;
    if (!(clip_low >= 0.0f && clip_low <= 1.0f) || !(clip_high >= 0.0f) || std::isinf(clip_high))
        return fail(RED_EINVAL, "red_policy: clip_low must be in 0..1 and clip_high finite and >= 0");
    if (std::isnan(kl_coef) || std::isinf(kl_coef) || std::isnan(grad_scale) || std::isinf(grad_scale))
        return fail(RED_EINVAL, "red_policy: kl_coef and grad_scale must be finite");
    if (kl_coef != 0.0f && rows > 0 && !ref_logp)
        return fail(RED_EINVAL, "red_policy: a KL term needs ref_logp");
    if (bad_ptr(stats, 4))
        return fail(RED_EINVAL, "red_policy: stats is NULL or not 4-byte aligned");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0)
        return zero_stats("red_policy: cudaMemsetAsync", stats, 4, s);
    if (bad_ptr(target, 8))
        return fail(RED_EINVAL, "red_policy: target is NULL or not 8-byte aligned");
    if (bad_ptr(old_logp, 4) || bad_opt(ref_logp, 4) || bad_ptr(adv, 4) || bad_opt(weight, 4))
        return fail(RED_EINVAL, "red_policy: old_logp or adv is NULL, or an input vector is not 4-byte aligned");
    if (bad_ptr(loss, 4) || bad_ptr(logp, 4))
        return fail(RED_EINVAL, "red_policy: loss or logp is NULL or not 4-byte aligned");
    return launch_policy(dtype, a,
                         PolicyArgs{target, old_logp, ref_logp, adv, weight, clip_low, clip_high, kl_coef,
                                    grad_scale, loss, logp, stats},
                         s);
}

int red_preference(int dtype, const void *x, int64_t rows, int64_t len, int64_t ld, float scale,
                   const int64_t *target, const int64_t *offsets, int64_t pairs, const float *ref_logp,
                   const float *weight, int kind, float beta, float margin, float smoothing, int average,
                   float grad_scale, float *loss, float *seq_logp, float *stats, float *work, void *dx, int64_t ldd,
                   red_stream_t stream)
{
    LogitRows a;
    const int st = logit_rows("red_preference", dtype, x, rows, len, ld, scale, dx, ldd, false, &a);
    if (st != RED_OK)
        return st;
    if (pairs < 0 || pairs > (int64_t(1) << 30))
        return fail(RED_EINVAL, "red_preference: pairs = %lld out of range", (long long)pairs);
    if (kind < RED_PREF_SIGMOID || kind > RED_PREF_SQUARED)
        return fail(RED_EINVAL, "red_preference: unknown kind %d", kind);
    if (!(beta > 0.0f) || std::isinf(beta) || std::isnan(margin) || std::isinf(margin))
        return fail(RED_EINVAL, "red_preference: beta must be positive and finite, margin finite");
    if (!(smoothing >= 0.0f && smoothing <= 0.5f) || (smoothing != 0.0f && kind != RED_PREF_SIGMOID))
        return fail(RED_EINVAL, "red_preference: smoothing must be in 0..0.5, and 0 unless the kind is sigmoid");
    if (std::isnan(grad_scale) || std::isinf(grad_scale))
        return fail(RED_EINVAL, "red_preference: grad_scale must be finite");
    if (bad_ptr(stats, 4))
        return fail(RED_EINVAL, "red_preference: stats is NULL or not 4-byte aligned");
    if (rows > 0 && bad_ptr(target, 8))
        return fail(RED_EINVAL, "red_preference: target is NULL or not 8-byte aligned");
    if ((rows > 0 || pairs > 0) && bad_ptr(work, 4))
        return fail(RED_EINVAL, "red_preference: work is NULL or not 4-byte aligned");
    if (pairs > 0 && (bad_ptr(offsets, 8) || bad_opt(ref_logp, 4) || bad_opt(weight, 4)))
        return fail(RED_EINVAL, "red_preference: offsets is NULL or not 8-byte aligned, or ref_logp or weight is "
                                "not 4-byte aligned");
    if (pairs > 0 && (bad_ptr(loss, 4) || bad_ptr(seq_logp, 4)))
        return fail(RED_EINVAL, "red_preference: loss or seq_logp is NULL or not 4-byte aligned");
    return launch_preference(dtype, a,
                             PreferenceArgs{pairs, target, offsets, ref_logp, weight, kind, average ? 1 : 0, beta,
                                            margin, smoothing, grad_scale, loss, seq_logp, stats, work, work + rows,
                                            work + 2 * rows, work + 3 * rows},
                             reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
