// Status, message and device check shared by the files that define C entry
// points (api.hip owns them).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/fp8lin.h"

namespace fp8lin {

// Clears the calling thread's message; every entry point starts with it.
void clear_error();
// Stores the message of a non-OK status (printf form) and returns the status.
fp8_status_t fail(fp8_status_t st, const char* fmt, ...);
fp8_status_t hip_fail(hipError_t e, const char* what);
// FP8_OK when the current device is a gfx950.
fp8_status_t check_device();
inline bool fmt_ok(fp8_fmt_t f) { return f == FP8_E4M3 || f == FP8_E5M2; }

}  // namespace fp8lin
