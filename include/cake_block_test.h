/*
 * cake_block_test.h -- entry points for tests of the block operators' bounded
 * waits and launch plans; no program needs them.
 */
#ifndef CAKE_BLOCK_TEST_H
#define CAKE_BLOCK_TEST_H

#include "cake_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Sets, for the calls of cake_block.h that this host thread makes from now on,
 * the limit of every wait in their kernels (1 to 1000000 microseconds), and
 * whether a part of what every CTA (of a pair, the first) of the gated block's
 * products and of the norm after dropout copies first never comes.  wait_limit_us = 0 with withhold = 0
 * restores the ordinary limit.  Anything else is CAKE_ERR_INVALID.  Every such
 * wait ends by its limit, the kernels return, and
 * cake_rmsnorm_device_status() gives CAKE_ERR_TIMEOUT.
 */
cake_status cake_block_wait_test(uint32_t wait_limit_us, int withhold);

/*
 * The plan of cake_dropout_norm_fwd (backward = 0) or _bwd for a shape and a
 * number of staged tensors (2, or 3 of the backward with dh): vectors of 8
 * columns of a thread, lanes of a row of part of a warp (32: none), warps of a
 * row, row groups, stages, CTAs, rows of a CTA, bytes of the threads' column sums, and bytes of shared memory.  Host
 * only.
 */
cake_status cake_dropout_norm_plan(const cake_shape *shape, int tensors, int backward, int64_t plan[9]);

#ifdef __cplusplus
}
#endif

#endif /* CAKE_BLOCK_TEST_H */
