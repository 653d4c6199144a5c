// Host pieces that every source file of the C ABI shares: how a refused
// launch is reported.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/gemv.h"

namespace gemvapi {

// GEMV_SUCCESS, or GEMV_ERROR_LAUNCH_FAILURE with `err` kept for
// gemv_last_hip_error (defined in gemv_api.hip).
__attribute__((visibility("hidden"))) gemv_status_t finish(hipError_t err);

}  // namespace gemvapi
