// Host helpers shared by the files that define C entry points.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>

#include <initializer_list>

#include "../../include/moe.h"

namespace moe {

constexpr size_t WS_ALIGN = 256;  // alignment of a workspace and of its regions

// Sets the thread's error text and returns s.
moe_status fail(moe_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
moe_status hip_status(hipError_t e, const char* what);
moe_status check_shape(const moe_shape* s);
moe_status check_rule(const moe_shape& s, const moe_gate_rule* r);

inline bool aligned(const void* p, size_t bytes) { return (uintptr_t)p % bytes == 0; }

// Memory of an argument; none where it is NULL
struct Span {
  const void* p;
  size_t bytes;
};
inline bool overlap(const Span& a, const Span& b) {
  return a.p && b.p && a.bytes && b.bytes && (uintptr_t)a.p < (uintptr_t)b.p + b.bytes && (uintptr_t)b.p < (uintptr_t)a.p + a.bytes;
}
// No output shares memory with an input or another output, the workspace being one of them.
inline moe_status check_outputs(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
  for (const Span* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Span* other = o + 1; other != outputs.end(); ++other)
      if (overlap(*o, *other)) return fail(MOE_ERR_INVALID_ARG, "two outputs, or an output and the workspace, share memory");
    for (const Span& in : inputs)
      if (overlap(*o, in)) return fail(MOE_ERR_INVALID_ARG, "an output or the workspace shares memory with an input");
  }
  return MOE_OK;
}

}  // namespace moe
