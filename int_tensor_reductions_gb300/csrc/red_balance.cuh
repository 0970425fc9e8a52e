// red_balance.cuh -- what the balance loss's kernels and its entry share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "red.h"

namespace red {

struct BalanceArgs {
    const void *x;
    int64_t rows, ldx;
    int experts;
    const int64_t *ids;
    int k;
    const uint8_t *live;  // NULL: all
    float coef, z_coef, grad_scale;
    int64_t *counts;
    float *prob, *stats;
    void *dx;             // NULL: no gradient
    int64_t ldd;
    unsigned *tick;       // workspace
    float *part;
};

int launch_balance(int dtype, BalanceArgs a, int kind, cudaStream_t s);

}  // namespace red
