// mgs_status.hpp — status codes and argument helpers shared by the C entry
// points (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mgs {

// Records a failed HIP call for mgs_last_hip_error; MGS_OK or MGS_ERR_HIP.
int hip_status(hipError_t e);

// Compute units of the current device.
int device_cus();

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace mgs
