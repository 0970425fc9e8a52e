// red_distill.cu -- distillation from a teacher's top logits (red_distill):
// the row kernel with a teacher warp, then the totals over rows.
#include "red_loss_rows.cuh"

namespace red {
namespace {

__global__ void __launch_bounds__(TOTAL_NT)
distill_total_kernel(int64_t rows, DistillArgs p, double *part, unsigned *tick)
{
    pdl_enter();
    total_rows<2>(rows, [&](int64_t r, double (&v)[2]) {
        v[0] += p.loss[r];
        v[1] += p.weight ? p.weight[r] : 1.0f;
    }, p.stats, part, tick);
}

}  // namespace

int launch_distill(int dtype, const LogitRows &a, const DistillArgs &p, cudaStream_t s)
{
    int st = launch_loss_rows(dtype, a, p, p.k, s);
    if (st != RED_OK)
        return st;
    Workspace ws;
    st = get_workspace(&ws);
    if (st != RED_OK)
        return st;
    const cudaError_t e = launch_pdl(distill_total_kernel, dim3(total_ctas(a.rows)), dim3(TOTAL_NT), s, a.rows, p,
                                     static_cast<double *>(ws.part), ws.tick);
    count_launches(1);
    return cuda_fail(e != cudaSuccess ? e : cudaGetLastError(), "red_distill launch");
}
}  // namespace red
