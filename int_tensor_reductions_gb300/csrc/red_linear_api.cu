// red_linear_api.cu -- the extern "C" entry points of red_linear_logprob and its
// backward (declared and documented in red.h): argument checks before any
// launch.
#include "red_linear.cuh"

using namespace red;

namespace {

constexpr int64_t MAX_ROWS = int64_t(1) << 24;  // rows and columns of tiles are 32-bit coordinates
constexpr int64_t MAX_DIM = int64_t(1) << 20;
constexpr int64_t MAX_LOGITS = int64_t(1) << 46;  // tiles are counted in 32 bits
constexpr int64_t MAX_STRIDE = int64_t(1) << 36;

bool bad_ptr(const void *p, uintptr_t align) { return !p || ((uintptr_t)p) % align != 0; }
bool bad_opt(const void *p, uintptr_t align) { return p && ((uintptr_t)p) % align != 0; }

int check_sizes(const char *who, int64_t rows, int64_t dim, int64_t vocab)
{
    if (rows < 0 || rows > MAX_ROWS || dim < 1 || dim > MAX_DIM || vocab < 1 || vocab > MAX_ROWS)
        return fail(RED_EINVAL, "%s: rows = %lld, dim = %lld, vocab = %lld out of range", who, (long long)rows,
                    (long long)dim, (long long)vocab);
    if (rows > MAX_LOGITS / vocab)
        return fail(RED_EINVAL, "%s: rows * vocab = %lld * %lld is over 2^46", who, (long long)rows, (long long)vocab);
    return RED_OK;
}

// A matrix that tensor maps describe.
int check_matrix(const char *who, const char *name, const void *p, int64_t rows, int64_t dim, int64_t ld)
{
    if (bad_ptr(p, 16))
        return fail(RED_EINVAL, "%s: %s is NULL or not 16-byte aligned", who, name);
    if (rows > 1 && (ld < dim || ld > MAX_STRIDE || ld % 8 != 0))
        return fail(RED_EINVAL, "%s: %s's row stride %lld must be a multiple of 8 elements and >= dim = %lld", who, name,
                    (long long)ld, (long long)dim);
    return RED_OK;
}

int check_work(const char *who, const void *work, int64_t bytes, int64_t needed)
{
    if (bad_ptr(work, 256))
        return fail(RED_EINVAL, "%s: work is NULL or not 256-byte aligned", who);
    if (bytes < needed)
        return fail(RED_EINVAL, "%s: work holds %lld bytes, %lld are needed", who, (long long)bytes, (long long)needed);
    return RED_OK;
}

// The checks that forward and backward share.
int linear_args(const char *who, LinearArgs *a)
{
    if (a->dtype != RED_F16 && a->dtype != RED_BF16)
        return fail(RED_EINVAL, "%s: dtype %d is not RED_F16 or RED_BF16", who, a->dtype);
    int st = check_sizes(who, a->rows, a->dim, a->vocab);
    if (st != RED_OK)
        return st;
    if (!(a->scale >= 1e-30f && a->scale <= 1e30f))
        return fail(RED_EINVAL, "%s: scale must be in 1e-30..1e30", who);
    if ((st = check_matrix(who, "weight", a->weight, a->vocab, a->dim, a->ldw)) != RED_OK)
        return st;
    if (a->vocab == 1)  // a single row's stride is never used, but a map wants one
        a->ldw = (a->dim + 7) / 8 * 8;
    if (a->rows == 0)
        return RED_OK;
    if ((st = check_matrix(who, "hidden", a->hidden, a->rows, a->dim, a->ldh)) != RED_OK)
        return st;
    if (a->rows == 1)
        a->ldh = (a->dim + 7) / 8 * 8;
    if (bad_ptr(a->target, 8))
        return fail(RED_EINVAL, "%s: target is NULL or not 8-byte aligned", who);
    return RED_OK;
}

}  // namespace

extern "C" {

int64_t red_linear_work_bytes(int64_t rows, int64_t dim, int64_t vocab, int grad)
{
    const int st = check_sizes("red_linear_work_bytes", rows, dim, vocab);
    if (st != RED_OK)
        return st;
    return linear_work(nullptr, rows, dim, vocab, grad != 0).bytes;
}

int red_linear_logprob(int dtype, const void *hidden, int64_t rows, int64_t dim, int64_t ldh, const void *weight,
                       int64_t vocab, int64_t ldw, float scale, const int64_t *target, float *logp, float *lse,
                       void *work, int64_t work_bytes, red_stream_t stream)
{
    const char *who = "red_linear_logprob";
    LinearArgs a = {dtype, hidden, rows, dim, ldh, weight, vocab, ldw, scale, target};
    int st = linear_args(who, &a);
    if (st != RED_OK || rows == 0)
        return st;
    if (bad_ptr(logp, 4) || bad_ptr(lse, 4))
        return fail(RED_EINVAL, "%s: logp or lse is NULL or not 4-byte aligned", who);
    if ((st = check_work(who, work, work_bytes, linear_work(nullptr, rows, dim, vocab, false).bytes)) != RED_OK)
        return st;
    return launch_linear_logprob(a, logp, lse, work, reinterpret_cast<cudaStream_t>(stream));
}

int red_linear_logprob_grad(int dtype, const void *hidden, int64_t rows, int64_t dim, int64_t ldh,
                            const void *weight, int64_t vocab, int64_t ldw, float scale, const int64_t *target,
                            const float *lse, const float *dlogp, const float *dlse, void *dhidden, int64_t ldd,
                            void *dweight, int64_t lddw, void *work, int64_t work_bytes, red_stream_t stream)
{
    const char *who = "red_linear_logprob_grad";
    LinearArgs a = {dtype, hidden, rows, dim, ldh, weight, vocab, ldw, scale, target};
    int st = linear_args(who, &a);
    if (st != RED_OK)
        return st;
    if (!dweight && !dhidden && rows > 0)
        return fail(RED_EINVAL, "%s: neither dhidden nor dweight is wanted", who);
    if (dweight) {
        if ((st = check_matrix(who, "dweight", dweight, vocab, dim, lddw)) != RED_OK)
            return st;
        if (vocab == 1)
            lddw = a.ldw;
        if (dweight == weight || dweight == hidden)
            return fail(RED_EINVAL, "%s: dweight overlaps an input", who);
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {
        if (!dweight)
            return RED_OK;
        return cuda_fail(cudaMemset2DAsync(dweight, (size_t)lddw * 2, 0, (size_t)dim * 2, (size_t)vocab, s),
                         "red_linear_logprob_grad: cudaMemset2DAsync");
    }
    if (dhidden) {
        if ((st = check_matrix(who, "dhidden", dhidden, rows, dim, ldd)) != RED_OK)
            return st;
        if (dhidden == weight || dhidden == dweight)
            return fail(RED_EINVAL, "%s: dhidden overlaps another matrix", who);
        if (dhidden == hidden && rows > 1 && ldd != ldh)
            return fail(RED_EINVAL, "%s: a gradient in place of hidden needs its row stride", who);
    }
    if (bad_ptr(lse, 4) || bad_ptr(dlogp, 4) || bad_opt(dlse, 4))
        return fail(RED_EINVAL, "%s: lse or dlogp is NULL, or a vector is not 4-byte aligned", who);
    if ((st = check_work(who, work, work_bytes, linear_work(nullptr, rows, dim, vocab, true).bytes)) != RED_OK)
        return st;
    return launch_linear_logprob_grad(a, lse, dlogp, dlse, dhidden, ldd, dweight, lddw, work, s);
}

}  // extern "C"
