// red_distill.cu -- distillation from a teacher's top logits (red_distill).
#include "red_loss_rows.cuh"

namespace red {

int launch_distill(int dtype, const LogitRows &a, const DistillArgs &p, cudaStream_t s)
{
    return launch_loss_rows(dtype, a, p, p.k, s);
}

}  // namespace red
