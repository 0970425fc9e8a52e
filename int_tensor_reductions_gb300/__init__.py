"""GB300-native fp32 / int32 axis reductions.

Python binding of libred.so (C ABI in ``include/red.h``): the functions below
carry the C entry points' names and only marshal arguments (torch tensors to
device pointers, sizes and the current CUDA stream); every step of every
reduction runs in the library's CUDA kernels.  There is no CPU fallback: if
libred.so is missing or CUDA is unavailable, the calls raise.

    red_full(op, x, out=None)                      op in "sum", "max", "min"
    red_rows(op, x, accum=False, out=None)         x: (rows, len) fp32
    red_rows_ragged(op, x, offsets, accum=False, out=None)
    red_colprod(x, out=None)                       x: (R, C) of any column element type
    red_cols(op, x, out=None)                      column sum / max / min / prod (x may be a
                                                   row-strided view: the C call red_cols_ld)
    red_full_typed / red_rows_typed                 full / per-row ops for every element type
    red_full_stats(x, out=None)                    sum, max, min, sum|x| in one read
    red_rows_stats(x, out=None)                    the same per row, out: (rows, 4)
    red_rows_thread(op, x, accum=False, out=None)  one thread per row, the page's fold order
    red_full_noalloc(op, x, out)                   red_full without any device allocation

Losses over rows of logits (float32, float16 or bfloat16), with their gradients:

    red_logprob(x, target)                         (log-probabilities, log-sum-exp) per row
    red_logprob_grad(x, target, lse, dlogp)        its backward
    red_distill(x, ids, vals)                      from a teacher's top logits
    red_policy(x, target, old_logp, adv)           clipped policy loss with a KL term
    red_preference(x, target, offsets)             pairs of packed sequences

The same from hidden states and the vocabulary's weights (float16 or bfloat16), without the logits:

    red_linear_logprob(hidden, weight, target)     (log-probabilities, log-sum-exp) per row
    red_linear_logprob_grad(hidden, weight, target, lse, dlogp)   its backward

Root-mean-square norm of rows, with the residual's addition, and the balance loss of a router:

    red_rmsnorm(x, weight, residual=r)             (y, x + r, 1 / root mean square)
    red_rmsnorm_quant(x, weight, residual=r)       with y in 8 bits and scales
    red_rmsnorm_grad(dy, x, rstd, weight)          the backward
    red_balance(x, ids)                            counts, mean probabilities, loss, gradient

Every call takes an optional ``stream`` (default: the current stream of x's
device) and returns ``out``.  Calls on one device must be ordered (one
stream, or streams ordered by events): they share the library's workspace.
"""
from ._binding import (  # noqa: F401
    RED_BF16, RED_DISTILL_MAX_K, RED_EINVAL, RED_ECUDA, RED_ENOMEM, RED_F16, RED_F32, RED_I16, RED_I32, RED_KNOB_COLPROD_SPLITS,
    RED_KNOB_FULL_CTAS_PER_SM, RED_KNOB_RAGGED_GROUP, RED_KNOB_RAGGED_STAGED, RED_KNOB_ROWS_ALIGNED, RED_KNOB_ROWS_GROUP,
    RED_KNOB_COLS_LANES, RED_KNOB_LOSS_TRIES, RED_MAX, RED_MIN,
    RED_BALANCE_MAX_EXPERTS, RED_BALANCE_SIGMOID, RED_BALANCE_SOFTMAX, RED_QUANT_E4M3, RED_QUANT_I8, RED_RMSNORM_MAX_LEN,
    RED_PREF_HINGE, RED_PREF_SIGMOID, RED_PREF_SQUARED,
    RED_MODE_ATOMIC, RED_MODE_AUTO, RED_MODE_LAST_BLOCK, RED_MODE_TWO_PASS, RED_OK, RED_PROD, RED_SUM, RED_U16, RED_U32,
    RedError, lib, lib_path, red_colprod, red_cols, red_distill, red_full, red_full_noalloc, red_full_stats, red_full_typed, red_get_full_mode, red_get_knob, red_last_error, red_balance, red_launch_count, red_linear_logprob,
    red_linear_logprob_grad, red_logprob, red_logprob_grad, red_policy, red_preference,
    red_release_workspace, red_rmsnorm, red_rmsnorm_grad, red_rmsnorm_quant, red_rows, red_rows_ragged, red_rows_stats, red_rows_thread, red_rows_typed, red_set_full_mode, red_set_knob, red_version,
)
