// api_status.h -- the calling thread's last error, shared by the files of the C ABI.
#pragma once

#include "moe.h"

namespace moe {

// Sets moe_last_error() and returns s.
moe_status api_fail(moe_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
void api_clear();

}  // namespace moe
