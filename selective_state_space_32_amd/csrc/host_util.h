// Host helpers of the translation units that hold an operator's entry points and kernels together
// (gated.hip, layernorm.hip) and so need nothing of launch.h, which declares the same ones for the
// scan's: the calling thread's status and message, and alignment.
#pragma once

#include <cstddef>
#include <cstdint>

#include "ssmscan.h"

namespace ssmlib {

// The status and message of the calling thread's last failure (ssm_last_error); defined in
// ssmscan.hip.
int fail(int code, const char *fmt, ...);
int ok();

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace ssmlib
