// ssg_abi.hpp -- what the sources of the C ABI share.
#pragma once

#include <cstdarg>
#include <cstdio>

namespace ssg {

// Records `text` as this thread's last error and returns `status`.
int abi_fail(int status, const char* text);

// The same with a format.
__attribute__((format(printf, 2, 3))) inline int abi_failf(int status, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return abi_fail(status, buf);
}

}  // namespace ssg
