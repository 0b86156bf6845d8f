// What the host sides of librtlynx's headers share (internal).
#pragma once

#include <hip/hip_runtime.h>

#include "rtlynx.h"

#define RTL_API extern "C" __attribute__((visibility("default")))

namespace rtl {

// Checks that a gfx950 device is current and that `stream` (NULL: the null
// stream) belongs to it; sets *cus to its CU count.
rtl_status check_device(hipStream_t stream, int* cus = nullptr);

inline rtl_status from_hip(hipError_t e) { return e == hipSuccess ? RTL_OK : RTL_ERR_HIP; }

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

}  // namespace rtl
