// red_loss.cuh -- building blocks of the losses over rows of logits
// (red_logprob, red_distill, red_policy, red_preference).
//
// Every loss is a function of the scaled logits z = scale * x of a row
// through its log-softmax.  With s2 = scale * log2(e) a row is reduced to its
// maximum m and
//     l = sum_j 2^(x_j * s2 - M),   M = m * s2 rounded to fp32,
// one multiply-add and one exponential per element.  The rounding of M, m *
// s2 - M = lo, is a common factor 2^lo of every term, taken back out where a
// logarithm is formed:
//     logp_y = scale * (x_y - m) - (ln l - lo ln 2),
//     lse    = scale * m + (ln l - lo ln 2),
//     p_j    = 2^(x_j * s2 - M) / l.
// Beyond |M| = 2^24 (a row that is nothing but the type's lowest value, say,
// as an additive mask leaves it) lo would no longer be small, and products of
// x overflow; there the terms are 2^((x_j - m) * s2), difference first.
// Partial (m, l) pairs combine by rescaling to the larger maximum, from one
// rounded M to the other; where no logit is finite m = -inf and l = 0.
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
    float s2;          // scale * log2(e), rounded
    float r_hi, r_lo;  // s2 / scale in two floats
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

constexpr float FAR = 16777216.0f;  // 2^24: the largest |M| of the multiply-add form

// The multiply-add form does for the maximum m (m * s2 = m2; not for a NaN).
__device__ __forceinline__ bool is_near(float m2) { return fabsf(m2) <= FAR; }

// Factor of a sum under the maximum `from` when the maximum becomes `to`; f2, t2:
// their products with s2, each rounded by itself (__fmul_rn).  The terms under a
// maximum are relative to its rounded product, so the exponent is the
// difference of those: with from * s2 - t2 in one multiply-add each partial sum
// would be off by 2^lo of its own maximum (log-probabilities near logits of
// 10^4 by 1.9e-4; 1e-6 as it is).  A far maximum is its product itself, unrounded.
__device__ __forceinline__ float soft_factor(float from, float f2, float to, float t2, float s2)
{
    float e = f2 - t2;
    if (!(fmaxf(fabsf(f2), fabsf(t2)) <= FAR)) {  // far, or -inf
        if (is_near(t2))
            e = fmaf(from, s2, -t2);
        else if (is_near(f2))
            e = fmaf(-to, s2, f2);
        else
            e = from == to ? 0.0f : (from - to) * s2;
    }
    return ex2(e);
}

// The largest of the lanes' values (no NaN), by the integer reduction: the
// bits of floats compare like integers once those of negative ones are turned
// around.
__device__ __forceinline__ float warp_max(float v)
{
    int b = __float_as_int(v + 0.0f);  // -0 becomes +0
    b ^= (b >> 31) & 0x7fffffff;
    b = __reduce_max_sync(0xffffffffu, b);
    return __int_as_float(b ^ ((b >> 31) & 0x7fffffff));
}

// The join over groups of W lanes that hold the same W values, in every lane:
// the maximum first, then one rescaling and the sum.
template <int W = 32>
__device__ __forceinline__ SoftStat soft_warp(SoftStat a, float s2)
{
    const float m = warp_max(a.m);
    float l = a.l * soft_factor(a.m, __fmul_rn(a.m, s2), m, __fmul_rn(m, s2), s2);
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1)
        l += __shfl_xor_sync(0xffffffffu, l, off);
    return SoftStat{m, l};
}

// A row's statistics as the losses use them.
struct RowStat {
    float m, m2;  // maximum, and M
    float l;      // the sum of terms
    float ln;     // logarithm of the sum relative to m itself
    bool far;     // terms are 2^((x - m) * s2)
    bool empty;   // every logit is -inf
};

__device__ __forceinline__ RowStat row_stat(const LogitRows &a, SoftStat t)
{
    RowStat s;
    s.m = t.m;
    s.l = t.l;
    s.m2 = t.m * a.s2;
    s.far = !is_near(s.m2);
    s.empty = t.m == NEG_INF && t.l == 0.0f;
    s.ln = logf(t.l);
    if (!s.far)
        s.ln = fmaf(-0.69314718f, fmaf(t.m, a.s2, -s.m2), s.ln);
    return s;
}

// ------------------------------------------------------------------- sums

// A sum in two floats, s + c: each addition's rounding error is computed
// (Knuth's two-sum) and carried along, so that the order of a long sum costs
// nothing and 64-bit arithmetic, 1/64 of the fp32 rate here, is not needed.
struct Sum {
    float s = 0.0f, c = 0.0f;

    __device__ __forceinline__ void add(float x)
    {
        const float t = s + x, z = t - s;
        c += (s - (t - z)) + (x - z);
        s = t;
    }
    __device__ __forceinline__ void add(const Sum &o)
    {
        add(o.s);
        c += o.c;
    }
    __device__ __forceinline__ void join_warp()
    {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            add(Sum{__shfl_xor_sync(0xffffffffu, s, off), __shfl_xor_sync(0xffffffffu, c, off)});
    }
    __device__ __forceinline__ float value() const { return isfinite(s) ? s + c : s; }
};

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
    const float e = expf(d);
    return e - (isinf(e) ? 0.0f : d + 1.0f);  // e^inf - inf is infinite
}

enum : int { ROW_END = 0, ROW_OUT = 1, ROW_LIVE = 2 };  // past the last row, out of the loss, in it

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
// or zeros throughout.  fc is 1 unless `far`.
struct RowGrad {
    float fa, fb, fc, mul, cy;
    int y;
    bool zero, far;
};

// mul * 2^(...) = c * p_j.
__device__ __forceinline__ RowGrad grad_of_stat(const LogitRows &a, const RowStat &t, float c)
{
    RowGrad g;
    g.far = t.far;
    g.fa = t.far ? 1.0f : a.s2;
    g.fb = t.far ? -t.m : -t.m2;
    g.fc = t.far ? a.s2 : 1.0f;
    g.mul = c / t.l;
    g.cy = 0.0f;
    g.y = -1;
    g.zero = t.empty;
    return g;
}

// c * ([j == y] - p_j).
__device__ __forceinline__ RowGrad grad_of_target(const LogitRows &a, const RowStat &t, int y, float c)
{
    RowGrad g = grad_of_stat(a, t, -c);
    g.cy = c;
    g.y = y;
    g.zero = t.empty || c == 0.0f;
    return g;
}

// Each loss below gives the kernels
//   STATS    whether a row's statistics come from its logits;
//   TEACHER  whether it has a list of teacher entries per row;
//   GRADIENT whether it can have a gradient;
//   TOTALS   how many sums over rows it has: total() adds a row's terms,
//            stats is where they go;
//   TAIL     whether something remains when all rows are done: the totals, or
//            tail();
//   load()   the row's entry (its logits are still intact): issues loads and
//            uses none of their values, so that a later settle() may be the
//            first to wait for them;
//   settle() whether the row takes part;
//   touch()  the load of the target's logit, its value not used either;
//   skip()   the row's scalar results when it takes no part;
//   grad()   the row's gradient from entry and statistics (any thread);
//   write()  the row's scalar results (one thread).

struct LogprobArgs {
    static constexpr bool STATS = true, TEACHER = false, GRADIENT = false;
    static constexpr bool TAIL = false;
    static constexpr int TOTALS = 0;
    const int64_t *target;
    float *logp, *lse;
    SoftStat *stat;  // statistics of rows [0, stat_rows) that take part, for their gradient
    int64_t stat_rows;

    __device__ void load(int64_t r, RowEntry &e) const
    {
        e.r = r;
        e.target = target[r];
    }
    __device__ void settle(const LogitRows &a, RowEntry &e) const
    {
        e.state = valid_id(e.target, a.len) ? ROW_LIVE : ROW_OUT;
    }
    template <int DT>
    __device__ void touch(const LogitRows &a, RowEntry &e) const
    {
        e.xy = load_bits<DT>(a.x, e.r * a.ld + e.target);
    }
    __device__ void skip(int64_t r) const { logp[r] = lse[r] = 0.0f; }
    template <int DT>
    __device__ RowGrad grad(const LogitRows &, const RowEntry &, const RowStat &, float) const { return RowGrad{}; }
    template <int DT>
    __device__ void write(const LogitRows &a, const RowEntry &e, const RowStat &t) const
    {
        logp[e.r] = t.empty ? NEG_INF : (Elem<DT>::widen(e.xy) - t.m) * a.scale - t.ln;
        lse[e.r] = t.empty ? NEG_INF : fmaf(a.scale, t.m, t.ln);
        if (e.r < stat_rows)
            stat[e.r] = SoftStat{t.m, t.l};
    }
};

struct LogprobGradArgs {
    static constexpr bool STATS = false, TEACHER = false, GRADIENT = true;
    static constexpr bool TAIL = false;
    static constexpr int TOTALS = 0;
    const int64_t *target;
    const float *lse, *dlogp;
    const SoftStat *stat;  // the rows' statistics; NULL: lse alone is known
    int64_t rows;

    // From the last row to the first: the logits that the forward pass read
    // last are the ones still in L2.
    __device__ void load(int64_t r, RowEntry &e) const
    {
        r = rows - 1 - r;
        e.r = r;
        e.target = target[r];
        e.w = dlogp[r];
        e.f[0] = lse[r];
        if (stat) {
            const SoftStat s = stat[r];
            e.f[1] = s.m;
            e.f[2] = s.l;
        }
    }
    __device__ void settle(const LogitRows &a, RowEntry &e) const
    {
        e.state = valid_id(e.target, a.len) && e.w != 0.0f && e.f[0] != NEG_INF ? ROW_LIVE : ROW_OUT;
    }
    template <int DT>
    __device__ void touch(const LogitRows &, RowEntry &) const {}
    __device__ void skip(int64_t) const {}
    // From the statistics as every loss forms it.  From lse, which its own
    // rounding leaves off by up to 2^-24 |lse|, and each probability by as much:
    // p_j = 2^(x_j * s2 - lse * s2 / scale), the same rounding of s2 in both
    // products; what the second one rounds away goes into the factor.  Far
    // from zero: 2^((scale x_j - lse) log2 e), the difference in one rounding.
    template <int DT>
    __device__ RowGrad grad(const LogitRows &a, const RowEntry &e, const RowStat &, float) const
    {
        const float n = e.f[0], c = e.w * a.scale;
        if (stat) {
            RowStat t{};
            t.m = e.f[1];
            t.l = e.f[2];
            t.m2 = t.m * a.s2;
            t.far = !is_near(t.m2);
            return grad_of_target(a, t, (int)e.target, c);
        }
        const float hi = n * a.r_hi, lo = fmaf(n, a.r_lo, fmaf(n, a.r_hi, -hi));
        RowGrad g;
        g.far = !is_near(hi);
        g.fa = g.far ? a.scale : a.s2;
        g.fb = g.far ? -n : -hi;
        g.fc = g.far ? LOG2E : 1.0f;
        g.mul = g.far ? -c : -c * ex2(-lo);
        g.cy = c;
        g.y = (int)e.target;
        g.zero = false;
        return g;
    }
    template <int DT>
    __device__ void write(const LogitRows &, const RowEntry &, const RowStat &) const {}
};

struct PolicyTerms {
    float loss;   // before the weight
    float drift;  // the KL estimate e^d - d - 1
    float clipped;
    float dlogp;
};

struct PolicyArgs {
    static constexpr bool STATS = true, TEACHER = false, GRADIENT = true;
    static constexpr bool TAIL = true;
    static constexpr int TOTALS = 4;
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
        // a ratio that overflowed, or of two tokens ruled out, times no advantage
        // is no gain, not a NaN; one of a NaN is
        const float free = A == 0.0f && (ratio == ratio || lp == old) ? 0.0f : ratio * A;
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
    __device__ void settle(const LogitRows &a, RowEntry &e) const
    {
        e.state = valid_id(e.target, a.len) && e.w != 0.0f ? ROW_LIVE : ROW_OUT;
    }
    template <int DT>
    __device__ void touch(const LogitRows &a, RowEntry &e) const
    {
        e.xy = load_bits<DT>(a.x, e.r * a.ld + e.target);
    }
    __device__ void skip(int64_t r) const { logp[r] = loss[r] = 0.0f; }
    template <int DT>
    __device__ float row_logp(const LogitRows &a, const RowEntry &e, const RowStat &t) const
    {
        return (Elem<DT>::widen(e.xy) - t.m) * a.scale - t.ln;
    }
    template <int DT>
    __device__ RowGrad grad(const LogitRows &a, const RowEntry &e, const RowStat &t, float) const
    {
        const PolicyTerms q = terms(row_logp<DT>(a, e, t), e.f[0], e.f[1], e.f[2]);
        return grad_of_target(a, t, (int)e.target, e.w * q.dlogp * gscale * a.scale);
    }
    template <int DT>
    __device__ void write(const LogitRows &a, const RowEntry &e, const RowStat &t) const
    {
        float p = NEG_INF, v = 0.0f;
        if (!t.empty) {
            p = row_logp<DT>(a, e, t);
            v = e.w * terms(p, e.f[0], e.f[1], e.f[2]).loss;
        }
        logp[e.r] = p;
        loss[e.r] = v;
    }
    __device__ void total(int64_t r, int len, Sum (&v)[TOTALS]) const
    {
        const float w = weight ? weight[r] : 1.0f, p = __ldcg(logp + r);
        if (!valid_id(target[r], len) || w == 0.0f)
            return;
        v[0].add(__ldcg(loss + r));
        v[3].add(w);
        if (p == NEG_INF)  // no ratio or drift to speak of
            return;
        const PolicyTerms q = terms(p, old_logp[r], ref_logp ? ref_logp[r] : 0.0f, adv[r]);
        v[1].add(w * q.drift);
        v[2].add(w * q.clipped);
    }
};

// Sum over groups of G lanes, in every lane; all lanes of the warp call it.
template <int G>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v)
{
    if constexpr (G == 32)
        return warp_max(v);
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// Teacher entries of a row in shared memory: k ids, then 3 * k floats.
struct TeacherRow {
    int *id;    // column, -1: no entry
    float *q;   // probability
    float *lq;  // its logarithm
    float *x;   // the student's logit
    float mass;   // sum of q (in the warp that prepared the row)
    bool repeat;  // an id comes more than once

    __device__ TeacherRow(void *base, int k)
    {
        id = static_cast<int *>(base);
        q = reinterpret_cast<float *>(id + k);
        lq = q + k;
        x = lq + k;
        mass = 0.0f;
        repeat = false;
    }
};

struct DistillArgs {
    static constexpr bool STATS = true, TEACHER = true, GRADIENT = true;
    static constexpr bool TAIL = true;
    static constexpr int TOTALS = 2;
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
    __device__ void settle(const LogitRows &, RowEntry &e) const { e.state = e.w != 0.0f ? ROW_LIVE : ROW_OUT; }
    template <int DT>
    __device__ void touch(const LogitRows &, RowEntry &) const {}
    __device__ void skip(int64_t r) const { loss[r] = 0.0f; }
    template <int DT>
    __device__ RowGrad grad(const LogitRows &a, const RowEntry &e, const RowStat &t, float Q) const
    {
        return grad_of_stat(a, t, e.w * gscale * a.scale * Q);
    }
    template <int DT>
    __device__ void write(const LogitRows &, const RowEntry &, const RowStat &) const {}

    // The three steps below are for groups of G lanes, a row each; all lanes
    // of the warp take part, those of rows out of the loss (`live` false) too.

    // Teacher probabilities of a row.
    template <int DT, int G>
    __device__ void prepare(const LogitRows &a, int64_t r, bool live, TeacherRow &s) const
    {
        const int gl = threadIdx.x & (G - 1);
        // Ids that come twice are looked for with a hash table in the space of
        // the floats, filled to two thirds at most; they are rare, and what
        // they cost is left to patch().
        const int size = 1 << (31 - __clz(3 * k));
        int *const table = reinterpret_cast<int *>(s.q);
        for (int i = gl; i < size; i += G)
            table[i] = -1;
        for (int i = gl; i < k; i += G) {
            const int64_t id = live ? ids[r * k + i] : -1;
            s.id[i] = valid_id(id, a.len) ? (int)id : -1;
        }
        __syncwarp();
        bool twice = false;
        for (int i = gl; i < k; i += G) {
            const int id = s.id[i];
            if (id < 0)
                continue;
            for (unsigned h = (unsigned)id * 2654435761u >> 7;; ++h) {
                const int was = atomicCAS(&table[h & (size - 1)], -1, id);
                twice = twice || was == id;
                if (was == -1 || was == id)
                    break;
            }
        }
        const unsigned any = __ballot_sync(0xffffffffu, twice);
        s.repeat = (any >> (threadIdx.x & 31 & ~(G - 1)) & (G == 32 ? 0xffffffffu : (1u << (G & 31)) - 1u)) != 0;
        float vmax = NEG_INF;
        for (int i = gl; i < k; i += G) {
            const int id = s.id[i];
            const float v = id >= 0 ? load_any(vdtype, vals, r * k + i) : NEG_INF;
            s.lq[i] = v;
            s.x[i] = id >= 0 ? load_elem<DT>(a.x, r * a.ld + id) : 0.0f;
            vmax = fmaxf(vmax, v);
        }
        // log q = scale * (v - base) - norm: from the largest value, or with the
        // normaliser that is given, in one rounding each, whatever the values' size
        float base = 0.0f, norm;
        if (lse) {
            norm = live ? lse[r] : 0.0f;
        } else {
            vmax = group_max<G>(fmaxf(vmax, NEG_INF));
            base = vmax == NEG_INF ? 0.0f : vmax;
            float sum = 0.0f;
            for (int i = gl; i < k; i += G)
                sum += expf((s.lq[i] - base) * a.scale);
            sum = group_sum<G>(sum);
            norm = vmax == NEG_INF && sum == 0.0f ? 0.0f : logf(sum);
        }
        float Q = 0.0f;
        for (int i = gl; i < k; i += G) {
            const float lq = fmaf(s.lq[i] - base, a.scale, -norm);
            const float q = s.id[i] < 0 ? 0.0f : expf(lq);
            s.lq[i] = lq;
            s.q[i] = q;
            Q += q;
        }
        s.mass = group_sum<G>(Q);
        __syncwarp();
    }
    // The row's loss, from the student's statistics.
    template <int G>
    __device__ void finish(const LogitRows &a, const RowEntry &e, const RowStat &t, const TeacherRow &s) const
    {
        const int gl = threadIdx.x & (G - 1);
        const bool on = e.state == ROW_LIVE && !t.empty;
        float v = 0.0f;
        if (on)
            for (int i = gl; i < k; i += G)
                if (s.q[i] != 0.0f)
                    v += s.q[i] * (s.lq[i] - ((s.x[i] - t.m) * a.scale - t.ln));
        v = group_sum<G>(v);
        if (gl == 0 && e.state == ROW_LIVE)
            loss[e.r] = on ? v * e.w : 0.0f;
    }
    // The teacher's columns of the gradient once more, after the rest of the
    // columns [begin, end) is written: g_id = mul 2^(...) - c q.  An id that
    // comes more than once is written by its first entry.
    template <int DT, int G>
    __device__ void patch(const LogitRows &a, const RowEntry &e, const RowGrad &g, const TeacherRow &s, int begin,
                          int end) const
    {
        const float c = e.w * gscale * a.scale;
        for (int i = threadIdx.x & (G - 1); i < k; i += G) {
            const int id = s.id[i];
            if (id < begin || id >= end)
                continue;
            float q = s.q[i];
            if (s.repeat) {
                q = 0.0f;
                bool first = true;
                for (int j = 0; j < k; ++j)
                    if (s.id[j] == id) {
                        first = first && j >= i;
                        q += s.q[j];
                    }
                if (!first)
                    continue;
            }
            store_elem<DT>(a.dx, e.r * a.ldd + id, g.mul * ex2(fmaf(s.x[i], g.fa, g.fb) * g.fc) - c * q);
        }
    }
    __device__ void total(int64_t r, int, Sum (&v)[TOTALS]) const
    {
        v[0].add(__ldcg(loss + r));
        v[1].add(weight ? weight[r] : 1.0f);
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
