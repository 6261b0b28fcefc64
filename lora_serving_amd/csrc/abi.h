// What the files that implement the C ABI share: argument checks and error reports.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mlora.h"

namespace mlora {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// MLORA_OK, or MLORA_ERR_HIP with the failure's text kept for mlora_last_error().
mlora_status hip_status(hipError_t e, const char *where = "launch");

}  // namespace mlora
