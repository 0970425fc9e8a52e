// red_linear.cuh -- log-probabilities of tokens from hidden states and the
// vocabulary's weights, without the logits (red_linear_logprob and its
// backward): what the translation units of the kernels and of the entry share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "red.h"
#include "red_internal.h"

namespace red {

// Device-side facts of a call, first in its workspace.
struct LinearHead {
    int live;      // rows that take part
    float unit;    // what the coefficients were divided by (gradients)
};

// Workspace of a call: rows that take part, packed, and what the passes hand on.
struct LinearWork {
    LinearHead *head;
    int *pos;           // rows: place among the packed rows, -1: none
    int *idx;           // packed: row
    int *target;        // packed: target
    void *hidden;       // packed hidden states, `padded` rows of `ld` elements, zeros behind the last
    float2 *part;       // packed x slots: (maximum of z / scale, sum)   (forward)
    float *at_target, *by_p, *lse2;  // packed: g at the target, coefficient of p, lse (gradients)
    void *piece;        // padded x piece: gradient by the logits (gradients)
    float *dhidden;     // splits x padded x dim4 sums            (gradients)
    int64_t padded, ld, dim4;
    int64_t slots;      // of part, per row
    int64_t piece_cols;
    int few;            // few rows: 16, 32, 64 or 128 columns, and piece is vocab x few
    int splits;         // shares of dh along the vocabulary
    int64_t bytes;
};

struct LinearArgs {
    int dtype;
    const void *hidden;
    int64_t rows, dim, ldh;
    const void *weight;
    int64_t vocab, ldw;
    float scale;
    const int64_t *target;
};

LinearWork linear_work(void *base, int64_t rows, int64_t dim, int64_t vocab, bool grad);

int launch_linear_logprob(const LinearArgs &a, float *logp, float *lse, void *work, cudaStream_t s);
int launch_linear_logprob_grad(const LinearArgs &a, const float *lse, const float *dlogp, const float *dlse,
                               void *dhidden, int64_t ldd, void *dweight, int64_t lddw, void *work, cudaStream_t s);

}  // namespace red
