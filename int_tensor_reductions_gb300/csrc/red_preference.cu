// red_preference.cu -- the preference loss of pairs of packed sequences: the
// row kernels of the log-probabilities and of their gradient around one
// kernel that reduces the packed tokens to sequences and pairs.
//
// One CTA per pair sums the log-probabilities of its two sequences, half of
// the threads each (in two floats and a fixed order: a sequence of thousands
// of tokens adds values of a few nats, and the loss depends on the difference
// of two such sums), forms u = beta * (gain of the chosen - gain of the
// rejected) - margin, the loss of u and its derivative, and writes each
// token's share of it.  The CTA that finishes last folds the totals over
// pairs.  It is bound by latency: three loads that wait for one another and
// two barriers, 4 us.
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
        t.du = u < 1.0f ? -1.0f : 0.0f;
    } else {
        const float off = (u - 0.5f) / p.beta;
        t.loss = off * off;
        t.du = 2.0f * off / p.beta;
    }
    return t;
}

__global__ void __launch_bounds__(NT) pair_kernel(int64_t rows, int len, PreferenceArgs p, unsigned *tick)
{
    pdl_enter();
    __shared__ Sum s[4 * NW];
    __shared__ int s_n[NW];
    __shared__ bool s_last;
    const int tid = threadIdx.x, side = tid / HALF;
    const int64_t pair = blockIdx.x;
    int64_t lo[2], hi[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t q = pair + i * p.pairs;
        // offsets outside [0, rows] are clamped, so no row outside is touched
        lo[i] = min(max(p.offsets[q], (int64_t)0), rows);
        hi[i] = min(max(p.offsets[q + 1], lo[i]), rows);
    }
    const float w = p.weight ? p.weight[pair] : 1.0f;
    const float ref0 = p.ref_logp ? p.ref_logp[pair] : 0.0f, ref1 = p.ref_logp ? p.ref_logp[pair + p.pairs] : 0.0f;
    Sum v;
    int n = 0;
    for (int64_t t = (side ? lo[1] : lo[0]) + tid % HALF; t < (side ? hi[1] : hi[0]); t += HALF) {
        const int64_t y = p.target[t];
        const float logp = p.logp[t], lse = p.lse[t];
        if (valid_id(y, len) && lse != NEG_INF) {
            v.add(logp);
            ++n;
        }
    }
    v.join_warp();
    n = __reduce_add_sync(0xffffffffu, n);
    if (tid % 32 == 0) {
        s[tid / 32] = v;
        s_n[tid / 32] = n;
    }
    __syncthreads();
    Sum sum[2];
    float count[2] = {1.0f, 1.0f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int total = 0;
#pragma unroll
        for (int k = 0; k < NW / 2; ++k) {
            sum[i].add(s[i * NW / 2 + k]);
            total += s_n[i * NW / 2 + k];
        }
        if (p.average) {
            count[i] = fmaxf((float)total, 1.0f);
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
    // rows before the first sequence and after the last belong to no loss
    if (pair == 0)
        for (int64_t r = tid; r < lo[0]; r += NT)
            p.dlogp[r] = 0.0f;
    if (pair == p.pairs - 1)
        for (int64_t r = hi[1] + tid; r < rows; r += NT)
            p.dlogp[r] = 0.0f;
    const float c = w == 0.0f ? 0.0f : (side ? -w : w) * t.du * p.beta * p.gscale / (side ? count[1] : count[0]);
    for (int64_t r = (side ? lo[1] : lo[0]) + tid % HALF; r < (side ? hi[1] : hi[0]); r += HALF)
        p.dlogp[r] = c;
    if (tid == 0) {
        p.loss[pair] = w == 0.0f ? 0.0f : w * t.loss;
        p.seq_logp[pair] = sum[0].value();
        p.seq_logp[pair + p.pairs] = sum[1].value();
        p.u[pair] = u;
        __threadfence();
        s_last = atomicAdd(tick, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last)
        return;
    __threadfence();
    Sum all[4];
    for (int64_t q = tid; q < p.pairs; q += NT) {
        const float wq = p.weight ? p.weight[q] : 1.0f;
        if (wq == 0.0f)
            continue;
        const float uq = __ldcg(p.u + q);
        all[0].add(__ldcg(p.loss + q));
        all[1].add(wq * uq);
        all[2].add(uq > 0.0f ? wq : 0.0f);
        all[3].add(wq);
    }
    cta_totals<4, NT>(all, s, p.stats);
    if (tid == 0)
        *tick = 0;
}

}  // namespace

int launch_preference(int dtype, const LogitRows &a, const PreferenceArgs &p, cudaStream_t s)
{
    int st = RED_OK;
    if (p.pairs == 0) {  // nothing to compare: no loss, a zero gradient
        cudaError_t e = cudaMemsetAsync(p.stats, 0, 4 * sizeof(float), s);
        if (e == cudaSuccess && a.rows > 0)
            e = cudaMemsetAsync(p.dlogp, 0, a.rows * sizeof(float), s);
        if (e != cudaSuccess)
            return cuda_fail(e, "red_preference: cudaMemsetAsync");
    } else {
        Workspace ws;
        st = get_workspace(&ws);
        if (st == RED_OK && a.rows > 0)
            st = launch_logprob(dtype, a, LogprobArgs{p.target, p.logp, p.lse}, s);
        if (st != RED_OK)
            return st;
        const cudaError_t e =
            launch_pdl(pair_kernel, dim3((unsigned)p.pairs), dim3(NT), s, a.rows, a.len, p, ws.tick);
        count_launches(1);
        st = cuda_fail(e != cudaSuccess ? e : cudaGetLastError(), "red_preference launch");
    }
    if (st != RED_OK || !a.dx || a.rows == 0)
        return st;
    return launch_logprob_grad(dtype, a, LogprobGradArgs{p.target, p.lse, p.dlogp, a.rows}, s);
}

}  // namespace red
