// red_policy.cu -- clipped policy loss with a KL term (red_policy).
#include "red_loss_rows.cuh"

namespace red {

int launch_policy(int dtype, const LogitRows &a, const PolicyArgs &p, cudaStream_t s)
{
    return launch_loss_rows(dtype, a, p, 0, s);
}

}  // namespace red
