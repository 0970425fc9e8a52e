// red_rmsnorm_api.cu -- the extern "C" entry points of the root-mean-square norm
// (declared and documented in red.h): argument checks before any launch.
#include <cmath>

#include "red_rmsnorm.cuh"

using namespace red;

namespace {

constexpr int64_t MAX_ELEMS = int64_t(1) << 44;

uintptr_t elem_size(int dtype) { return dtype == RED_F32 ? 4 : 2; }
bool float_type(int dtype) { return dtype == RED_F32 || dtype == RED_F16 || dtype == RED_BF16; }

int check_types(const char *who, int dtype, int64_t rows, int64_t len, int wtype, const void *weight)
{
    if (!float_type(dtype))
        return fail(RED_EINVAL, "%s: dtype %d is not RED_F32, RED_F16 or RED_BF16", who, dtype);
    if (rows < 0 || rows > MAX_ELEMS / RED_RMSNORM_MAX_LEN || len < 1 || len > RED_RMSNORM_MAX_LEN)
        return fail(RED_EINVAL, "%s: rows = %lld, len = %lld out of range (len 1..%d)", who, (long long)rows,
                    (long long)len, RED_RMSNORM_MAX_LEN);
    if (wtype != dtype && wtype != RED_F32)
        return fail(RED_EINVAL, "%s: wtype %d is neither x's type nor RED_F32", who, wtype);
    if ((uintptr_t)weight % elem_size(wtype) != 0)
        return fail(RED_EINVAL, "%s: weight is not aligned to its element size", who);
    return RED_OK;
}

int check_matrix(const char *who, const char *name, const void *p, uintptr_t elem, int64_t rows, int64_t len, int64_t ld)
{
    if (!p || (uintptr_t)p % elem != 0)
        return fail(RED_EINVAL, "%s: %s is NULL or not aligned to its element size", who, name);
    if (rows > 1 && (ld < len || ld > MAX_ELEMS / rows))
        return fail(RED_EINVAL, "%s: %s's row stride %lld must be >= len = %lld and rows * stride in range", who, name,
                    (long long)ld, (long long)len);
    return RED_OK;
}

// Written rows may lie where read rows do, element on element, or nowhere near.
int check_over(const char *who, const char *name, const void *out, int64_t ldo, const void *in, int64_t ldi, int64_t rows)
{
    if (out && out == in && rows > 1 && ldo != ldi)
        return fail(RED_EINVAL, "%s: %s in place of an input needs its row stride", who, name);
    return RED_OK;
}

#define TRY(call)          \
    if ((st = (call)) != RED_OK) \
    return st

int forward(const char *who, int dtype, NormArgs &a, int64_t len, int wtype, int kind, cudaStream_t s)
{
    int st;
    TRY(check_types(who, dtype, a.rows, len, wtype, a.weight));
    if (!(a.eps >= 0.0f && a.eps <= 1e30f))
        return fail(RED_EINVAL, "%s: eps must be in 0..1e30", who);
    if (a.rows == 0)
        return RED_OK;
    const uintptr_t elem = elem_size(dtype);
    TRY(check_matrix(who, "x", a.x, elem, a.rows, len, a.ldx));
    TRY(check_matrix(who, kind ? "q" : "y", a.y, kind ? 1 : elem, a.rows, len, a.ldy));
    if (!a.residual != !a.total)
        return fail(RED_EINVAL, "%s: residual and total come together", who);
    if (a.residual) {
        TRY(check_matrix(who, "residual", a.residual, elem, a.rows, len, a.ldr));
        TRY(check_matrix(who, "total", a.total, elem, a.rows, len, a.ldt));
        TRY(check_over(who, "total", a.total, a.ldt, a.x, a.ldx, a.rows));
        TRY(check_over(who, "total", a.total, a.ldt, a.residual, a.ldr, a.rows));
        if (a.total == a.y)
            return fail(RED_EINVAL, "%s: total and the result overlap", who);
    }
    if (kind) {
        if (a.y == a.x || a.y == a.residual)
            return fail(RED_EINVAL, "%s: q overlaps an input", who);
    } else {
        TRY(check_over(who, "y", a.y, a.ldy, a.x, a.ldx, a.rows));
        TRY(check_over(who, "y", a.y, a.ldy, a.residual, a.ldr, a.rows));
    }
    if ((uintptr_t)a.rstd % 4 != 0)
        return fail(RED_EINVAL, "%s: rstd is not 4-byte aligned", who);
    a.len = (int)len;
    a.wide = wtype == RED_F32;
    a.inv_len = (float)(1.0 / (double)len);
    return dtype == RED_F32   ? rmsnorm_forward<RED_F32>(a, kind, s)
           : dtype == RED_F16 ? rmsnorm_forward<RED_F16>(a, kind, s)
                              : rmsnorm_forward<RED_BF16>(a, kind, s);
}

}  // namespace

extern "C" {

int red_rmsnorm(int dtype, const void *x, int64_t rows, int64_t len, int64_t ldx, const void *residual, int64_t ldr,
                int wtype, const void *weight, float eps, void *y, int64_t ldy, void *total, int64_t ldt, float *rstd,
                red_stream_t stream)
{
    NormArgs a = {};
    a.x = x, a.residual = residual, a.weight = weight, a.rows = rows, a.ldx = ldx, a.ldr = ldr, a.eps = eps;
    a.y = y, a.ldy = ldy, a.total = total, a.ldt = ldt, a.rstd = rstd;
    return forward("red_rmsnorm", dtype, a, len, wtype, 0, reinterpret_cast<cudaStream_t>(stream));
}

int red_rmsnorm_quant(int dtype, const void *x, int64_t rows, int64_t len, int64_t ldx, const void *residual,
                      int64_t ldr, int wtype, const void *weight, float eps, int kind, int64_t block, void *q,
                      int64_t ldq, float *scales, void *total, int64_t ldt, float *rstd, red_stream_t stream)
{
    const char *who = "red_rmsnorm_quant";
    if (kind != RED_QUANT_E4M3 && kind != RED_QUANT_I8)
        return fail(RED_EINVAL, "%s: unknown kind %d", who, kind);
    if (block != 0 && block != 32 && block != 64 && block != 128)
        return fail(RED_EINVAL, "%s: block = %lld is not 0, 32, 64 or 128", who, (long long)block);
    if (rows > 0 && (!scales || (uintptr_t)scales % 4 != 0))
        return fail(RED_EINVAL, "%s: scales is NULL or not 4-byte aligned", who);
    NormArgs a = {};
    a.x = x, a.residual = residual, a.weight = weight, a.rows = rows, a.ldx = ldx, a.ldr = ldr, a.eps = eps;
    a.y = q, a.ldy = ldq, a.total = total, a.ldt = ldt, a.rstd = rstd, a.scales = scales;
    if (block > 0 && block < len) {  // (else one scale per row, whichever it is called)
        a.block = (int)block;
        a.block_log2 = block == 32 ? 5 : block == 64 ? 6 : 7;
        a.blocks = (int)((len + block - 1) / block);
    } else {
        a.blocks = 1;
    }
    return forward(who, dtype, a, len, wtype, kind, reinterpret_cast<cudaStream_t>(stream));
}

int red_rmsnorm_grad(int dtype, const void *dy, int64_t lddy, const void *x, int64_t rows, int64_t len, int64_t ldx,
                     const float *rstd, int wtype, const void *weight, const void *dtotal, int64_t ldt, void *dx,
                     int64_t ldd, void *dweight, red_stream_t stream)
{
    const char *who = "red_rmsnorm_grad";
    int st;
    TRY(check_types(who, dtype, rows, len, wtype, weight));
    if ((uintptr_t)dweight % elem_size(wtype) != 0)
        return fail(RED_EINVAL, "%s: dweight is not aligned to its element size", who);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {
        if (!dweight)
            return RED_OK;
        return cuda_fail(cudaMemsetAsync(dweight, 0, (size_t)len * elem_size(wtype), s),
                         "red_rmsnorm_grad: cudaMemsetAsync");
    }
    const uintptr_t elem = elem_size(dtype);
    TRY(check_matrix(who, "dy", dy, elem, rows, len, lddy));
    TRY(check_matrix(who, "x", x, elem, rows, len, ldx));
    TRY(check_matrix(who, "dx", dx, elem, rows, len, ldd));
    if (dtotal)
        TRY(check_matrix(who, "dtotal", dtotal, elem, rows, len, ldt));
    TRY(check_over(who, "dx", dx, ldd, dy, lddy, rows));
    TRY(check_over(who, "dx", dx, ldd, x, ldx, rows));
    TRY(check_over(who, "dx", dx, ldd, dtotal, ldt, rows));
    if (!rstd || (uintptr_t)rstd % 4 != 0)
        return fail(RED_EINVAL, "%s: rstd is NULL or not 4-byte aligned", who);
    NormGradArgs a = {};
    a.dy = dy, a.x = x, a.weight = weight, a.dtotal = dtotal, a.rstd = rstd, a.rows = rows, a.ldy = lddy, a.ldx = ldx;
    a.ldt = ldt, a.ldd = ldd, a.dx = dx, a.dw = dweight, a.wtype = wtype;
    a.len = (int)len;
    a.wide = wtype == RED_F32;
    a.inv_len = (float)(1.0 / (double)len);
    return dtype == RED_F32   ? rmsnorm_backward<RED_F32>(a, s)
           : dtype == RED_F16 ? rmsnorm_backward<RED_F16>(a, s)
                              : rmsnorm_backward<RED_BF16>(a, s);
}

}  // extern "C"
