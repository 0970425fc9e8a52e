// red_rmsnorm_grad_f32.cu -- the root-mean-square norm's backward for f32 rows.
#define RED_RMSNORM_DT RED_F32
#define RED_RMSNORM_BACKWARD
#include "red_rmsnorm.cuh"
