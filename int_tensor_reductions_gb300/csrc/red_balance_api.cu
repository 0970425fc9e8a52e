// red_balance_api.cu -- the extern "C" entry point of the balance loss (declared
// and documented in red.h): argument checks before any launch.
#include <cmath>

#include "red_balance.cuh"
#include "red_internal.h"

using namespace red;

extern "C" int red_balance(int dtype, const void *x, int64_t rows, int64_t experts, int64_t ld, const int64_t *ids,
                           int64_t k, const uint8_t *live, int kind, float coef, float z_coef, float grad_scale,
                           int64_t *counts, float *prob, float *stats, void *dx, int64_t ldd, red_stream_t stream)
{
    const char *who = "red_balance";
    constexpr int64_t MAX_ELEMS = int64_t(1) << 44, MAX_ENTRIES = int64_t(1) << 31;
    if (dtype != RED_F32 && dtype != RED_F16 && dtype != RED_BF16)
        return fail(RED_EINVAL, "%s: dtype %d is not RED_F32, RED_F16 or RED_BF16", who, dtype);
    if (experts < 1 || experts > RED_BALANCE_MAX_EXPERTS || k < 1 || k > experts)
        return fail(RED_EINVAL, "%s: experts = %lld (1..%d) or k = %lld (1..experts) out of range", who,
                    (long long)experts, RED_BALANCE_MAX_EXPERTS, (long long)k);
    if (rows < 0 || rows >= MAX_ENTRIES / k)
        return fail(RED_EINVAL, "%s: rows = %lld out of range (rows * k < 2^31)", who, (long long)rows);
    if (kind != RED_BALANCE_SOFTMAX && kind != RED_BALANCE_SIGMOID)
        return fail(RED_EINVAL, "%s: unknown kind %d", who, kind);
    if (!std::isfinite(coef) || !std::isfinite(z_coef) || !std::isfinite(grad_scale))
        return fail(RED_EINVAL, "%s: coef, z_coef and grad_scale must be finite", who);
    if (kind == RED_BALANCE_SIGMOID && z_coef != 0.0f)
        return fail(RED_EINVAL, "%s: z_coef is of the softmax alone", who);
    if (!counts || (uintptr_t)counts % 8 != 0)
        return fail(RED_EINVAL, "%s: counts is NULL or not 8-byte aligned", who);
    if (!prob || (uintptr_t)prob % 4 != 0 || !stats || (uintptr_t)stats % 4 != 0)
        return fail(RED_EINVAL, "%s: prob or stats is NULL or not 4-byte aligned", who);
    const uintptr_t elem = dtype == RED_F32 ? 4 : 2;
    if (rows > 0) {
        if (!x || (uintptr_t)x % elem != 0)
            return fail(RED_EINVAL, "%s: x is NULL or not aligned to its element size", who);
        if (!ids || (uintptr_t)ids % 8 != 0)
            return fail(RED_EINVAL, "%s: ids is NULL or not 8-byte aligned", who);
        if ((uintptr_t)dx % elem != 0)
            return fail(RED_EINVAL, "%s: dx is not aligned to its element size", who);
        if (rows > 1 && (ld < experts || ld > MAX_ELEMS / rows || (dx && (ldd < experts || ldd > MAX_ELEMS / rows))))
            return fail(RED_EINVAL, "%s: a row stride is below experts = %lld or out of range", who, (long long)experts);
        if (dx == x && rows > 1 && ldd != ld)
            return fail(RED_EINVAL, "%s: a gradient in place needs x's row stride", who);
    }
    BalanceArgs a = {};
    a.x = x, a.rows = rows, a.ldx = ld, a.experts = (int)experts, a.ids = ids, a.k = (int)k, a.live = live;
    a.coef = coef, a.z_coef = z_coef, a.grad_scale = grad_scale, a.counts = counts, a.prob = prob, a.stats = stats;
    a.dx = dx, a.ldd = ldd;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {
        cudaError_t e = cudaMemsetAsync(counts, 0, (size_t)experts * 8, s);
        if (e == cudaSuccess)
            e = cudaMemsetAsync(prob, 0, (size_t)experts * 4, s);
        if (e == cudaSuccess)
            e = cudaMemsetAsync(stats, 0, 16, s);
        return cuda_fail(e, "red_balance: cudaMemsetAsync");
    }
    return launch_balance(dtype, a, kind, s);
}
