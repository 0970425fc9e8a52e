// red_rmsnorm_f32.cu -- the root-mean-square norm's kernels for f32 rows.
#define RED_RMSNORM_DT RED_F32
#include "red_rmsnorm.cuh"
