// red_loss.cu -- kernels of the losses over rows of logits.
//
// One CTA per row: pass 1 reduces the row to its softmax statistics, one
// thread (one warp for the distillation) turns them into the row's loss and
// the coefficient of its gradient, pass 2 reads the row again and writes the
// gradient.
#include "red_internal.h"
#include "red_loss.cuh"
#include "red_prims.cuh"

namespace red {
namespace {

constexpr int NT = 256;
constexpr int NW = NT / 32;

// Statistics of a row, in every thread.
template <int DT>
__device__ SoftStat row_stat(const void *row, int len, float s2, SoftStat *s_w)
{
    SoftStat t{NEG_INF, 0.0f};
    for (int j = threadIdx.x; j < len; j += NT) {
        const float v = load_elem<DT>(row, j);
        const float m = fmaxf(t.m, v), at = ref_of(m);
        t.l = t.l * ex2((t.m - at) * s2) + ex2((v - at) * s2);
        t.m = m;
    }
    t = soft_warp(t, s2);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        s_w[threadIdx.x >> 5] = t;
    __syncthreads();
    t = s_w[0];
    for (int w = 1; w < NW; ++w)
        t = soft_join(t, s_w[w], s2);
    return t;
}

template <int DT>
__device__ const void *row_ptr(const LogitRows &a, int64_t r)
{
    return static_cast<const typename Elem<DT>::T *>(a.x) + r * a.ld;
}
template <int DT>
__device__ void *grad_ptr(const LogitRows &a, int64_t r)
{
    return static_cast<typename Elem<DT>::T *>(a.dx) + r * a.ldd;
}

template <int DT>
__device__ void zero_row(void *g, int len)
{
    for (int j = threadIdx.x; j < len; j += NT)
        store_elem<DT>(g, j, 0.0f);
}

// g_j = c * ([j == y] - 2^((x_j - m) * s2) / l); nothing finite: zeros.
template <int DT>
__device__ void target_grad(const void *row, void *g, int len, SoftStat t, float s2, float c, int y)
{
    if (t.m == NEG_INF)
        return zero_row<DT>(g, len);
    const float a = -c / t.l;
    for (int j = threadIdx.x; j < len; j += NT) {
        float v = a * ex2((load_elem<DT>(row, j) - t.m) * s2);
        if (j == y)
            v += c;
        store_elem<DT>(g, j, v);
    }
}

template <int DT>
__global__ void __launch_bounds__(NT) logprob_kernel(LogitRows a, LogprobArgs p)
{
    pdl_enter();
    __shared__ SoftStat s_w[NW];
    const float s2 = a.scale * LOG2E;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t y = p.target[r];
        float logp = 0.0f, lse = 0.0f;
        if (valid_id(y, a.len)) {
            const void *row = row_ptr<DT>(a, r);
            const SoftStat t = row_stat<DT>(row, a.len, s2, s_w);
            const float ln = logf(t.l);
            lse = t.m == NEG_INF && t.l == 0.0f ? NEG_INF : fmaf(a.scale, t.m, ln);
            logp = lse == NEG_INF ? NEG_INF : (load_elem<DT>(row, y) - t.m) * a.scale - ln;
        }
        if (threadIdx.x == 0) {
            p.logp[r] = logp;
            p.lse[r] = lse;
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(NT)
logprob_grad_kernel(LogitRows a, const int64_t *__restrict__ target, const float *__restrict__ lse,
                    const float *__restrict__ dlogp)
{
    pdl_enter();
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t y = target[r];
        const void *row = row_ptr<DT>(a, r);
        void *g = grad_ptr<DT>(a, r);
        const float n = lse[r], d = dlogp[r];
        if (!valid_id(y, a.len) || d == 0.0f || n == NEG_INF) {
            zero_row<DT>(g, a.len);
            continue;
        }
        const float c = d * a.scale;
        for (int j = threadIdx.x; j < a.len; j += NT) {
            float v = -c * ex2(fmaf(load_elem<DT>(row, j), a.scale, -n) * LOG2E);
            if (j == y)
                v += c;
            store_elem<DT>(g, j, v);
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(NT) policy_kernel(LogitRows a, PolicyArgs p)
{
    pdl_enter();
    __shared__ SoftStat s_w[NW];
    const float s2 = a.scale * LOG2E;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t y = p.target[r];
        const float w = p.weight ? p.weight[r] : 1.0f;
        const void *row = row_ptr<DT>(a, r);
        SoftStat t{NEG_INF, 0.0f};
        const bool live = valid_id(y, a.len) && w != 0.0f;
        float logp = 0.0f, loss = 0.0f, c = 0.0f;
        if (live) {
            const float xy = load_elem<DT>(row, y);
            t = row_stat<DT>(row, a.len, s2, s_w);
            if (t.m == NEG_INF && t.l == 0.0f) {
                logp = NEG_INF;
            } else {
                logp = (xy - t.m) * a.scale - logf(t.l);
                const PolicyTerms q = policy_terms(logp, p.old_logp[r], p.ref_logp ? p.ref_logp[r] : 0.0f,
                                                   p.ref_logp != nullptr, p.adv[r], p.clip_low, p.clip_high, p.kl);
                loss = w * q.loss;
                c = w * q.dlogp * p.gscale * a.scale;
            }
        }
        if (threadIdx.x == 0) {
            p.logp[r] = logp;
            p.loss[r] = loss;
        }
        if (a.dx) {
            if (t.m == NEG_INF && t.l == 0.0f)
                zero_row<DT>(grad_ptr<DT>(a, r), a.len);
            else
                target_grad<DT>(row, grad_ptr<DT>(a, r), a.len, t, s2, c, (int)y);
        }
    }
}

// Teacher probabilities of a row, by warp 0: s_id (-1: unused), s_q, s_lq
// (log q) and s_x (the student's logit); returns Q = sum q.
template <int DT>
__device__ float teacher_row(const LogitRows &a, const DistillArgs &p, int64_t r, const void *row, int *s_id,
                             float *s_q, float *s_lq, float *s_x)
{
    const int lane = threadIdx.x & 31;
    float vmax = NEG_INF;
    for (int i = lane; i < p.k; i += 32) {
        const int64_t id = p.ids[r * p.k + i];
        const bool ok = valid_id(id, a.len);
        const float v = ok ? load_any(p.vdtype, p.vals, r * p.k + i) * a.scale : NEG_INF;
        s_id[i] = ok ? (int)id : -1;
        s_lq[i] = v;
        s_x[i] = ok ? load_elem<DT>(row, id) : 0.0f;
        vmax = fmaxf(vmax, v);
    }
    float norm;
    if (p.lse) {
        norm = p.lse[r];
    } else {
        vmax = group_tree<OP_MAX, 32>(vmax);
        float s = 0.0f;
        for (int i = lane; i < p.k; i += 32)
            s += expf(s_lq[i] - ref_of(vmax));
        s = group_tree<OP_SUM, 32>(s);
        norm = vmax == NEG_INF && s == 0.0f ? 0.0f : vmax + logf(s);
    }
    float Q = 0.0f;
    for (int i = lane; i < p.k; i += 32) {
        const float lq = s_lq[i] - norm;
        const float q = s_id[i] < 0 ? 0.0f : expf(lq);
        s_lq[i] = lq;
        s_q[i] = q;
        Q += q;
    }
    return group_tree<OP_SUM, 32>(Q);
}

template <int DT>
__global__ void __launch_bounds__(NT) distill_kernel(LogitRows a, DistillArgs p)
{
    pdl_enter();
    __shared__ SoftStat s_w[NW];
    __shared__ int s_id[RED_DISTILL_MAX_K];
    __shared__ float s_q[RED_DISTILL_MAX_K], s_lq[RED_DISTILL_MAX_K], s_x[RED_DISTILL_MAX_K], s_Q;
    const float s2 = a.scale * LOG2E;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const float w = p.weight ? p.weight[r] : 1.0f;
        const void *row = row_ptr<DT>(a, r);
        void *g = a.dx ? grad_ptr<DT>(a, r) : nullptr;
        SoftStat t{NEG_INF, 0.0f};
        if (w != 0.0f) {
            if (threadIdx.x < 32) {
                const float Q = teacher_row<DT>(a, p, r, row, s_id, s_q, s_lq, s_x);
                if (threadIdx.x == 0)
                    s_Q = Q;
            }
            t = row_stat<DT>(row, a.len, s2, s_w);
        }
        const bool none = t.m == NEG_INF && t.l == 0.0f;
        if (threadIdx.x < 32) {
            float loss = 0.0f;
            if (!none) {
                const float ln = logf(t.l);
                for (int i = threadIdx.x; i < p.k; i += 32)
                    if (s_q[i] != 0.0f)
                        loss += s_q[i] * (s_lq[i] - ((s_x[i] - t.m) * a.scale - ln));
                loss = group_tree<OP_SUM, 32>(loss) * w;
            }
            if (threadIdx.x == 0)
                p.loss[r] = loss;
        }
        if (!g)
            continue;
        if (none) {
            zero_row<DT>(g, a.len);
            continue;
        }
        const float c = w * p.gscale * a.scale;
        const float A = c * s_Q / t.l;
        for (int j = threadIdx.x; j < a.len; j += NT)
            store_elem<DT>(g, j, A * ex2((load_elem<DT>(row, j) - t.m) * s2));
        __syncthreads();
        // the teacher's tokens once more, each id by its first entry
        for (int i = threadIdx.x; i < p.k; i += NT) {
            const int id = s_id[i];
            if (id < 0)
                continue;
            float q = 0.0f;
            bool first = true;
            for (int k = 0; k < p.k; ++k)
                if (s_id[k] == id) {
                    first = first && k >= i;
                    q += s_q[k];
                }
            if (first)
                store_elem<DT>(g, id, A * ex2((s_x[i] - t.m) * s2) - c * q);
        }
        __syncthreads();
    }
}

// Totals over rows, from what the row kernels left (one CTA, 64-bit sums in
// a fixed order).
constexpr int TOTAL_NT = 1024;

template <int N>
__device__ void cta_total(double (&v)[N], float *out)
{
    __shared__ double s[N][32];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        for (int off = 16; off > 0; off >>= 1)
            v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
        if ((threadIdx.x & 31) == 0)
            s[i][threadIdx.x >> 5] = v[i];
    }
    __syncthreads();
    if (threadIdx.x < N) {
        double t = 0.0;
        for (int w = 0; w < (int)blockDim.x / 32; ++w)
            t += s[threadIdx.x][w];
        out[threadIdx.x] = (float)t;
    }
}

__global__ void __launch_bounds__(TOTAL_NT) policy_total_kernel(int64_t rows, int len, PolicyArgs p)
{
    pdl_enter();
    double v[4] = {0.0, 0.0, 0.0, 0.0};
    for (int64_t r = threadIdx.x; r < rows; r += TOTAL_NT) {
        const float w = p.weight ? p.weight[r] : 1.0f;
        const float logp = p.logp[r];
        if (!valid_id(p.target[r], len) || w == 0.0f)
            continue;
        v[3] += w;
        if (logp == NEG_INF) {  // no ratio or drift to speak of; its loss may be infinite
            v[0] += p.loss[r];
            continue;
        }
        const PolicyTerms q = policy_terms(logp, p.old_logp[r], p.ref_logp ? p.ref_logp[r] : 0.0f,
                                           p.ref_logp != nullptr, p.adv[r], p.clip_low, p.clip_high, p.kl);
        v[0] += p.loss[r];
        v[1] += w * q.drift;
        v[2] += w * q.clipped;
    }
    cta_total(v, p.stats);
}

__global__ void __launch_bounds__(TOTAL_NT)
distill_total_kernel(int64_t rows, DistillArgs p)
{
    pdl_enter();
    double v[2] = {0.0, 0.0};
    for (int64_t r = threadIdx.x; r < rows; r += TOTAL_NT) {
        v[0] += p.loss[r];
        v[1] += p.weight ? p.weight[r] : 1.0f;
    }
    cta_total(v, p.stats);
}

unsigned row_ctas(int64_t rows, int sms)
{
    const int64_t cap = (int64_t)sms * 8;
    return (unsigned)(rows < cap ? rows : cap);
}

template <typename F>
int by_dtype(int dtype, F f)
{
    switch (dtype) {
    case RED_F32: return f(std::integral_constant<int, RED_F32>());
    case RED_F16: return f(std::integral_constant<int, RED_F16>());
    default: return f(std::integral_constant<int, RED_BF16>());
    }
}

}  // namespace

int launch_logprob(int dtype, const LogitRows &a, const LogprobArgs &p, cudaStream_t s)
{
    DeviceInfo di;
    const int st = device_info(&di);
    if (st != RED_OK)
        return st;
    return by_dtype(dtype, [&](auto dt) {
        const cudaError_t e = launch_pdl(logprob_kernel<dt()>, dim3(row_ctas(a.rows, di.sms)), dim3(NT), s, a, p);
        count_launches(1);
        return cuda_fail(e != cudaSuccess ? e : cudaGetLastError(), "red_logprob launch");
    });
}

int launch_logprob_grad(int dtype, const LogitRows &a, const int64_t *target, const float *lse, const float *dlogp,
                        cudaStream_t s)
{
    DeviceInfo di;
    const int st = device_info(&di);
    if (st != RED_OK)
        return st;
    return by_dtype(dtype, [&](auto dt) {
        const cudaError_t e = launch_pdl(logprob_grad_kernel<dt()>, dim3(row_ctas(a.rows, di.sms)), dim3(NT), s, a,
                                         target, lse, dlogp);
        count_launches(1);
        return cuda_fail(e != cudaSuccess ? e : cudaGetLastError(), "red_logprob_grad launch");
    });
}

int launch_policy(int dtype, const LogitRows &a, const PolicyArgs &p, cudaStream_t s)
{
    DeviceInfo di;
    const int st = device_info(&di);
    if (st != RED_OK)
        return st;
    return by_dtype(dtype, [&](auto dt) {
        cudaError_t e = launch_pdl(policy_kernel<dt()>, dim3(row_ctas(a.rows, di.sms)), dim3(NT), s, a, p);
        if (e == cudaSuccess)
            e = launch_pdl(policy_total_kernel, dim3(1), dim3(TOTAL_NT), s, a.rows, a.len, p);
        count_launches(2);
        return cuda_fail(e != cudaSuccess ? e : cudaGetLastError(), "red_policy launch");
    });
}

int launch_distill(int dtype, const LogitRows &a, const DistillArgs &p, cudaStream_t s)
{
    DeviceInfo di;
    const int st = device_info(&di);
    if (st != RED_OK)
        return st;
    return by_dtype(dtype, [&](auto dt) {
        cudaError_t e = launch_pdl(distill_kernel<dt()>, dim3(row_ctas(a.rows, di.sms)), dim3(NT), s, a, p);
        if (e == cudaSuccess)
            e = launch_pdl(distill_total_kernel, dim3(1), dim3(TOTAL_NT), s, a.rows, p);
        count_launches(2);
        return cuda_fail(e != cudaSuccess ? e : cudaGetLastError(), "red_distill launch");
    });
}

}  // namespace red
