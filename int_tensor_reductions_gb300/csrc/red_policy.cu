// red_policy.cu -- clipped policy loss with a KL term (red_policy): the row
// kernel, then the totals over rows from the log-probabilities it left.
#include "red_loss_rows.cuh"

namespace red {
namespace {

__global__ void __launch_bounds__(TOTAL_NT)
policy_total_kernel(int64_t rows, int len, PolicyArgs p, double *part, unsigned *tick)
{
    pdl_enter();
    total_rows<4>(rows, [&](int64_t r, double (&v)[4]) {
        const float w = p.weight ? p.weight[r] : 1.0f;
        if (!valid_id(p.target[r], len) || w == 0.0f)
            return;
        const float logp = p.logp[r];
        v[0] += p.loss[r];
        v[3] += w;
        if (logp == NEG_INF)  // no ratio or drift to speak of
            return;
        const PolicyTerms q = p.terms(logp, p.old_logp[r], p.ref_logp ? p.ref_logp[r] : 0.0f, p.adv[r]);
        v[1] += w * q.drift;
        v[2] += w * q.clipped;
    }, p.stats, part, tick);
}

}  // namespace

int launch_policy(int dtype, const LogitRows &a, const PolicyArgs &p, cudaStream_t s)
{
    int st = launch_loss_rows(dtype, a, p, 0, s);
    if (st != RED_OK)
        return st;
    Workspace ws;
    st = get_workspace(&ws);
    if (st != RED_OK)
        return st;
    const cudaError_t e = launch_pdl(policy_total_kernel, dim3(total_ctas(a.rows)), dim3(TOTAL_NT), s, a.rows, a.len, p,
                                     static_cast<double *>(ws.part), ws.tick);
    count_launches(1);
    return cuda_fail(e != cudaSuccess ? e : cudaGetLastError(), "red_policy launch");
}

}  // namespace red
