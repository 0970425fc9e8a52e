// red_logprob.cu -- log-probabilities of given columns of rows of logits, and
// their gradient (red_logprob, red_logprob_grad).
#include "red_loss_rows.cuh"

namespace red {

int launch_logprob(int dtype, const LogitRows &a, const LogprobArgs &p, cudaStream_t s)
{
    LogitRows rows = a;
    rows.dx = nullptr;  // the statistics alone
    return launch_loss_rows(dtype, rows, p, 0, s);
}

}  // namespace red
