// Status and message of the C ABI's entry points (defined in capi.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "w4a4.h"

namespace w4a4 {

// Sets the thread's message and returns st.
w4a4_status fail(w4a4_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the message.
w4a4_status ok();
w4a4_status hip_status(hipError_t e, const char* what);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace w4a4
