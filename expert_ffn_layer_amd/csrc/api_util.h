// Host helpers shared by the files that define C entry points.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>

#include "../../include/moe.h"

namespace moe {

constexpr size_t WS_ALIGN = 256;  // alignment of a workspace and of its regions

// Sets the thread's error text and returns s.
moe_status fail(moe_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
moe_status hip_status(hipError_t e, const char* what);
moe_status check_shape(const moe_shape* s);

}  // namespace moe
