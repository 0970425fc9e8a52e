// red_rmsnorm_f16.cu -- the root-mean-square norm's kernels for f16 rows.
#define RED_RMSNORM_DT RED_F16
#include "red_rmsnorm.cuh"
