/*
 * cake_step_test.h -- an entry point for tests of the training-step operators'
 * bounded waits; no program needs it.
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

#ifdef __cplusplus
}
#endif

#endif /* CAKE_STEP_TEST_H */
