// Error reporting of the C ABI layer: the calling thread's last message and
// the mapping of HIP errors to a status (defined in api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pc.h"

namespace pc {

// Stores the message of a failing call and returns its status.
pc_status fail(pc_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the message.
pc_status ok();
pc_status hip_status(hipError_t e, const char *what);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace pc
