// red_rmsnorm_bf16.cu -- the root-mean-square norm's kernels for bf16 rows.
#define RED_RMSNORM_DT RED_BF16
#include "red_rmsnorm.cuh"
