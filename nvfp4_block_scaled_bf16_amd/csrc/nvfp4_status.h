// nvfp4_status.h -- how the C ABI's translation units report: the thread's
// last error and the checks they share.  Not part of the public interface.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cstdarg>
#include <cstdio>
#include <string>

#include "nvfp4.h"

namespace nvfp4 {

inline thread_local std::string g_last_error;

inline nvfp4_status fail(nvfp4_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return st;
}

inline nvfp4_status ok() {
    g_last_error.clear();
    return NVFP4_OK;
}

inline nvfp4_status check_hip(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(NVFP4_EDEVICE, "%s: %s", what, hipGetErrorString(e));
    return NVFP4_OK;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace nvfp4
