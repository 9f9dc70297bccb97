// cake_step_device.cuh -- device pieces shared by the kernels of the
// training-step operators.
#pragma once

#include "../csrc/cake_device.cuh"

namespace cake {

// Records a status code.  The operators share one word for two codes: the
// larger one stays, so that an id outside its table (CAKE_ERR_INVALID, 1, whose
// outputs are defined) never hides a wait that ran out (CAKE_ERR_TIMEOUT, 5,
// whose outputs are not).
__device__ __forceinline__ void raise_status(int *status, int code)
{
    atomicMax(status, code);
}

} // namespace cake
