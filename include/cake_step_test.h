/*
 * cake_step_test.h -- entry points for tests of the training-step operators'
 * bounded waits and launch plans; no program needs them.
 */
#ifndef CAKE_STEP_TEST_H
#define CAKE_STEP_TEST_H

#include "cake_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Sets, for the calls of cake_step.h that this host thread makes from now on,
 * the limit of every wait in their kernels (1 to 1000000 microseconds), and
 * what never comes:
 *   withhold = 0  nothing: a wait may run out only by being too short;
 *   withhold = 1  a part of what every CTA of a sandwich norm stages first, and
 *                 the flag that the embedding gradient's zeroing CTAs wait for;
 *   withhold = 2  the same for the sandwich norm's first CTA alone (the others
 *                 of its cluster wait for its sums).
 * wait_limit_us = 0 with withhold = 0 restores the ordinary limit.  Anything
 * else is CAKE_ERR_INVALID.  Every such wait ends by its limit, the kernels
 * return, and cake_rmsnorm_device_status() gives CAKE_ERR_TIMEOUT.
 */
cake_status cake_step_wait_test(uint32_t wait_limit_us, int withhold);

/*
 * The plan of cake_sandwich_bwd for a shape and a number of staged tensors (3,
 * and one more each for an element gate and dh).  plan: the kernel's build
 * (16-byte vectors of a thread, whether rows span a cluster, room for a row's
 * warps, whether more than 12 consumer warps run, whether a thread takes half
 * a vector more), then CTAs of a cluster, rows of a stage, stages, and stages'
 * worth of rows of the largest CTA or cluster.  Host only.
 */
cake_status cake_sandwich_bwd_plan(const cake_shape *shape, int tensors, int plan[9]);

/* Whether the calls take two tensors of a shape to share memory.  Host only. */
int cake_step_rows_meet(const cake_shape *shape, const cake_tensor *a, const cake_tensor *b);

#ifdef __cplusplus
}
#endif

#endif /* CAKE_STEP_TEST_H */
