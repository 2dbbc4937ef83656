// What the two files of the C ABI share.
#pragma once

#include "../../include/scan.h"

#include <hip/hip_runtime.h>

namespace sca {
namespace api {

// SCAN_OK, or SCAN_EHIP with the error kept for scan_last_hip_error().
scan_status hip_status(hipError_t e);

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace api
}  // namespace sca
