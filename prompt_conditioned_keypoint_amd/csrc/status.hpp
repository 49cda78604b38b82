// status.hpp - the thread's error text and the status helpers of the C ABI
// sources (defined in api.hip).
#pragma once

#include "gkdhead.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gkd {

// Sets the thread's error text and returns s.
__attribute__((format(printf, 2, 3))) gkd_status fail(gkd_status s, const char* fmt, ...);
// Clears the thread's error text.
gkd_status ok();
// GKD_OK, or GKD_ERR_HIP with the runtime's text.
gkd_status hip_status(hipError_t e, const char* what);

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace gkd
