// red_logprob_grad.cu -- the gradient of log-probabilities by the logits, from
// the rows' log-sum-exp (red_logprob_grad): one pass, no statistics.
#include "red_loss_rows.cuh"

namespace red {

int launch_logprob_grad(int dtype, const LogitRows &a, const LogprobGradArgs &p, cudaStream_t s)
{
    return launch_loss_rows(dtype, a, p, 0, s);
}

}  // namespace red
