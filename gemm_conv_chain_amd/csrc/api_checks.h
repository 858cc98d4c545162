// api_checks.h -- what the C ABI's sources for serving share: the calling
// thread's error, and alignment.
#pragma once
#include <stdarg.h>
#include <stdio.h>

#include "../../include/fusedchain.h"
#include "fc_launch.h"

namespace fc {

inline fc_status fail(fc_status s, const char* fmt, ...)
{
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    return (fc_status)api_fail(s, msg);
}

inline fc_status done(hipError_t e, const char* what)
{
    if (e != hipSuccess) return fail(FC_E_HIP, "%s: %s", what, hipGetErrorString(e));
    return (fc_status)api_fail(FC_OK, "");
}

inline bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace fc
