// red_preference.cu -- the preference loss of pairs of packed sequences: the
// row kernels of the log-probabilities and of their gradient around one
// kernel that reduces the packed tokens to sequences and pairs.
//
// A pair's kernel sums the log-probabilities of its two sequences (in two
// floats and a fixed order: a sequence of thousands of tokens adds values of a
// few nats, and the loss depends on the difference of two such sums), forms
// u = beta * (gain of the chosen - gain of the rejected) - margin, the loss of
// u and its derivative, and writes each token's share of it; the last to
// finish folds the totals over pairs.  It is bound by latency (three loads
// that wait for one another and two barriers, 4 us), so where rows and pairs
// are few the last CTA of the log-probabilities does the same, a warp per
// pair (190 x 16384 f32: 13.9 -> 13.3 us for the whole call, 200 x 20000 bf16: 12.8
// -> 12.0, and 2.4 us less of the host's time).
#include "red_internal.h"
#include "red_loss_rows.cuh"

namespace red {
namespace {

constexpr int NT = 512;
constexpr int NW = NT / 32, HALF = NT / 2;

struct PairTerms {
    float loss, du;
};

__device__ PairTerms pair_terms(const PreferenceArgs &p, float u)
{
    PairTerms t;
    if (p.kind == RED_PREF_SIGMOID) {
        // -(1 - e) log sigma(u) - e log sigma(-u); log sigma through
        // log1p(e^-|u|), which neither overflows nor loses small values
        const float e = p.smoothing, soft = log1pf(expf(-fabsf(u)));
        t.loss = (1.0f - e) * (soft + fmaxf(-u, 0.0f));
        if (e != 0.0f)  // (u may be infinite: a token that the policy rules out)
            t.loss += e * (soft + fmaxf(u, 0.0f));
        t.du = e - 1.0f / (1.0f + expf(u));
        if (u != u)
            t.loss = u;
    } else if (p.kind == RED_PREF_HINGE) {
        t.loss = u < 1.0f ? 1.0f - u : (u != u ? u : 0.0f);
        t.du = u < 1.0f ? -1.0f : (u != u ? u : 0.0f);
    } else {
        const float off = (u - 0.5f) / p.beta;
        t.loss = off * off;
        t.du = 2.0f * off / p.beta;
    }
    return t;
}

// Rows of the two sequences of a pair.
struct PairRows {
    int64_t lo[2], hi[2];
};

__device__ PairRows pair_rows(const PreferenceArgs &p, int64_t pair, int64_t rows)
{
    PairRows b;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t q = pair + i * p.pairs;
        // offsets outside [0, rows] are clamped, so no row outside is touched
        b.lo[i] = min(max(p.offsets[q], (int64_t)0), rows);
        b.hi[i] = min(max(p.offsets[q + 1], b.lo[i]), rows);
    }
    return b;
}

// What rows [lo, hi), every `step`th from `first`, add to their sequence.
__device__ void add_rows(const PreferenceArgs &p, int64_t lo, int64_t hi, int first, int step, int len, Sum &v, int &n)
{
    for (int64_t t = lo + first; t < hi; t += step) {
        const int64_t y = p.target[t];
        const float logp = __ldcg(p.logp + t), lse = __ldcg(p.lse + t);
        if (valid_id(y, len) && lse != NEG_INF) {
            v.add(logp);
            ++n;
        }
    }
}

// The pair's loss from its sequences' sums and counts, written by the thread
// for which `write`; returns the gradient by each token's log-probability.
__device__ float2 pair_loss(const PreferenceArgs &p, int64_t pair, Sum (&sum)[2], const int (&n)[2], float w,
                            float ref0, float ref1, bool write)
{
    float count[2] = {1.0f, 1.0f};
    if (p.average) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            count[i] = fmaxf((float)n[i], 1.0f);
            const float mean = sum[i].s / count[i];
            sum[i] = Sum{mean, (fmaf(-mean, count[i], sum[i].s) + sum[i].c) / count[i]};
        }
    }
    Sum gain = sum[0];
    gain.add(Sum{-sum[1].s, -sum[1].c});
    gain.add(-ref0);
    gain.add(ref1);
    const float u = fmaf(p.beta, gain.value(), -p.margin);
    PairTerms t{0.0f, 0.0f};
    if (w != 0.0f)
        t = pair_terms(p, u);
    if (write) {
        p.loss[pair] = w == 0.0f ? 0.0f : w * t.loss;
        p.seq_logp[pair] = sum[0].value();
        p.seq_logp[pair + p.pairs] = sum[1].value();
        p.u[pair] = u;
    }
    const float c = w == 0.0f ? 0.0f : w * t.du * p.beta * p.gscale;
    return make_float2(c / count[0], -c / count[1]);
}

// Rows before the first sequence and after the last belong to no loss.
__device__ void clear_outside(const PreferenceArgs &p, int64_t pair, const PairRows &b, int64_t rows, int first,
                              int step)
{
    if (pair == 0)
        for (int64_t r = first; r < b.lo[0]; r += step)
            p.dlogp[r] = 0.0f;
    if (pair == p.pairs - 1)
        for (int64_t r = b.hi[1] + first; r < rows; r += step)
            p.dlogp[r] = 0.0f;
}

template <int T>
__device__ void pair_totals(const PreferenceArgs &p, Sum *s)
{
    Sum all[4];
    for (int64_t q = threadIdx.x; q < p.pairs; q += T) {
        const float wq = p.weight ? p.weight[q] : 1.0f;
        if (wq == 0.0f)
            continue;
        const float uq = __ldcg(p.u + q);
        all[0].add(__ldcg(p.loss + q));
        all[1].add(wq * uq);
        all[2].add(uq > 0.0f ? wq : 0.0f);
        all[3].add(wq);
    }
    cta_totals<4, T>(all, s, p.stats);
}

// A CTA per pair, half of the threads per sequence.
__global__ void __launch_bounds__(NT) pair_kernel(int64_t rows, int len, PreferenceArgs p, unsigned *tick)
{
    pdl_enter();
    __shared__ Sum s[4 * NW];
    __shared__ int s_n[NW];
    __shared__ bool s_last;
    const int tid = threadIdx.x, side = tid / HALF;
    const int64_t pair = blockIdx.x;
    const PairRows b = pair_rows(p, pair, rows);
    const float w = p.weight ? p.weight[pair] : 1.0f;
    const float ref0 = p.ref_logp ? p.ref_logp[pair] : 0.0f, ref1 = p.ref_logp ? p.ref_logp[pair + p.pairs] : 0.0f;
    const int64_t lo = side ? b.lo[1] : b.lo[0], hi = side ? b.hi[1] : b.hi[0];
    Sum v;
    int n = 0;
    add_rows(p, lo, hi, tid % HALF, HALF, len, v, n);
    v.join_warp();
    n = __reduce_add_sync(0xffffffffu, n);
    if (tid % 32 == 0) {
        s[tid / 32] = v;
        s_n[tid / 32] = n;
    }
    __syncthreads();
    Sum sum[2];
    int count[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < NW / 2; ++k) {
            sum[i].add(s[i * NW / 2 + k]);
            count[i] += s_n[i * NW / 2 + k];
        }
    const float2 c = pair_loss(p, pair, sum, count, w, ref0, ref1, tid == 0);
    for (int64_t r = lo + tid % HALF; r < hi; r += HALF)
        p.dlogp[r] = side ? c.y : c.x;
    clear_outside(p, pair, b, rows, tid, NT);
    if (tid == 0) {
        __threadfence();
        s_last = atomicAdd(tick, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last)
        return;
    __threadfence();
    pair_totals<NT>(p, s);
    if (tid == 0)
        *tick = 0;
}

// The log-probabilities of few rows, and then their pairs.
struct PreferenceForward : LogprobArgs {
    static constexpr bool TAIL = true;
    PreferenceArgs p;

    template <int T>
    __device__ void tail(int64_t rows, int len, Sum *s) const
    {
        const int lane = threadIdx.x & 31;
        for (int64_t pair = threadIdx.x / 32; pair < p.pairs; pair += T / 32) {
            const PairRows b = pair_rows(p, pair, rows);
            const float w = p.weight ? p.weight[pair] : 1.0f;
            const float ref0 = p.ref_logp ? p.ref_logp[pair] : 0.0f;
            const float ref1 = p.ref_logp ? p.ref_logp[pair + p.pairs] : 0.0f;
            Sum sum[2];
            int n[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 2; ++i)
                add_rows(p, b.lo[i], b.hi[i], lane, 32, len, sum[i], n[i]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                sum[i].join_warp();
                n[i] = __reduce_add_sync(0xffffffffu, n[i]);
            }
            const float2 c = pair_loss(p, pair, sum, n, w, ref0, ref1, lane == 0);
            for (int64_t r = b.lo[0] + lane; r < b.hi[0]; r += 32)
                p.dlogp[r] = c.x;
            for (int64_t r = b.lo[1] + lane; r < b.hi[1]; r += 32)
                p.dlogp[r] = c.y;
            clear_outside(p, pair, b, rows, lane, 32);
        }
        __syncthreads();
        pair_totals<T>(p, s);
    }
};

// Pairs up to which the few-row kernel's last CTA does them all, a warp each.
// (The same by the last CTA of short rows was measured and left out: 1000 x
// 1000 bf16 in 30 pairs 15.3 us against 10.7, the totals of 1000 x 1024 bf16
// policy rows 8.9 against 7.5.)
constexpr int64_t TAIL_PAIRS = FEW_NW;

template <int DT>
int launch_forward(const LogitRows &a, const PreferenceForward &f, cudaStream_t s, bool *taken)
{
    DeviceInfo di;
    const int st = device_info(&di);
    if (st != RED_OK)
        return st;
    return launch_few<DT>(a, f, 0, s, di, taken);
}

}  // namespace

int launch_preference(int dtype, const LogitRows &a, const PreferenceArgs &p, cudaStream_t s)
{
    int st = RED_OK;
    const bool grad = a.dx && a.rows > 0;
    Workspace ws;
    if (grad || p.pairs > 0)
        st = get_workspace(&ws);
    if (st != RED_OK)
        return st;
    // The gradient takes the rows' statistics as the forward pass left them in
    // the workspace: lse in 32 bits would put the probabilities off, by 3e-5 at
    // |lse| = 1000, and make each of them 1 in a row of nothing but the type's
    // lowest value.
    SoftStat *const stat = static_cast<SoftStat *>(ws.part);
    const int64_t room = WS_PART_BYTES / sizeof(SoftStat);
    const int64_t kept = !grad ? 0 : (a.rows < room ? a.rows : room);
    if (p.pairs == 0) {  // nothing to compare: no loss, a zero gradient
        cudaError_t e = cudaMemsetAsync(p.stats, 0, 4 * sizeof(float), s);
        if (e == cudaSuccess && a.rows > 0)
            e = cudaMemsetAsync(p.dlogp, 0, a.rows * sizeof(float), s);
        if (e != cudaSuccess)
            return cuda_fail(e, "red_preference: cudaMemsetAsync");
    } else {
        const LogprobArgs forward{p.target, p.logp, p.lse, stat, kept};
        bool taken = false;
        if (a.rows > 0 && p.pairs <= TAIL_PAIRS) {
            LogitRows rows = a;
            rows.dx = nullptr;
            PreferenceForward f;
            static_cast<LogprobArgs &>(f) = forward;
            f.p = p;
            switch (dtype) {
            case RED_F32: st = launch_forward<RED_F32>(rows, f, s, &taken); break;
            case RED_F16: st = launch_forward<RED_F16>(rows, f, s, &taken); break;
            default: st = launch_forward<RED_BF16>(rows, f, s, &taken); break;
            }
        }
        if (st != RED_OK)
            return st;
        if (!taken) {
            if (a.rows > 0)
                st = launch_logprob(dtype, a, forward, s);
            if (st != RED_OK)
                return st;
            const cudaError_t e =
                launch_pdl(pair_kernel, dim3((unsigned)p.pairs), dim3(NT), s, a.rows, a.len, p, ws.tick);
            count_launches(1);
            st = cuda_fail(e != cudaSuccess ? e : cudaGetLastError(), "red_preference launch");
        }
    }
    // Rows beyond the workspace's room (2^21) have their statistics formed again,
    // as many at a time.
    for (int64_t lo = 0; grad && st == RED_OK && lo < a.rows; lo += room) {
        const int64_t size = dtype == RED_F32 ? 4 : 2;
        LogitRows part = a;
        part.rows = a.rows - lo < room ? a.rows - lo : room;
        part.x = static_cast<const char *>(a.x) + lo * a.ld * size;
        part.dx = static_cast<char *>(a.dx) + lo * a.ldd * size;
        const int64_t *const target = p.target + lo;
        if (lo > 0)
            st = launch_logprob(dtype, part, LogprobArgs{target, p.logp + lo, p.lse + lo, stat, part.rows}, s);
        if (st == RED_OK)
            st = launch_logprob_grad(dtype, part,
                                     LogprobGradArgs{target, p.lse + lo, p.dlogp + lo, stat, part.rows}, s);
    }
    return st;
}

}  // namespace red
