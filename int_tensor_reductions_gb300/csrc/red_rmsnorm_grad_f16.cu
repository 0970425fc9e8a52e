// red_rmsnorm_grad_f16.cu -- the root-mean-square norm's backward for f16 rows.
#define RED_RMSNORM_DT RED_F16
#define RED_RMSNORM_BACKWARD
#include "red_rmsnorm.cuh"
