// Failure text and log lines for the library's other translation units: both
// are defined beside the C ABI's own (mscl.hip), so that
// mscl_last_error_string() and MSCL_LOG cover every entry point.
#pragma once

#include "../../include/mscl.h"

namespace mscl {

// Keeps `msg` as the calling thread's last error and returns `s`.
__attribute__((visibility("hidden"))) mscl_status_t record_failure(mscl_status_t s, const char* msg);

// A line on stderr when MSCL_LOG is at least `level`.
__attribute__((visibility("hidden"))) void log_text(int level, const char* msg);

}  // namespace mscl
