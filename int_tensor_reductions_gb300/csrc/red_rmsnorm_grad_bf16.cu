// red_rmsnorm_grad_bf16.cu -- the root-mean-square norm's backward for bf16 rows.
#define RED_RMSNORM_DT RED_BF16
#define RED_RMSNORM_BACKWARD
#include "red_rmsnorm.cuh"
