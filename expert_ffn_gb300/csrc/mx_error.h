// mx_error.h -- the calling thread's error message (mx_last_error_string).
#pragma once

#include "mx_moe.h"

namespace mx {

// Records a printf-style message and returns `s`.
mx_status fail(mx_status s, const char *fmt, ...);

}  // namespace mx
