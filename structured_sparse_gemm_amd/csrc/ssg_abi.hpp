// ssg_abi.hpp -- what the sources of the C ABI share.
#pragma once

namespace ssg {

// Records `text` as this thread's last error and returns `status`.
int abi_fail(int status, const char* text);

}  // namespace ssg
