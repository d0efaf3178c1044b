// Host-side argument checks shared by the files that implement the C ABI.
#pragma once

#include "internal.h"

namespace moe {

// Records the calling thread's error message and returns `st`.
moe_status fail(moe_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
moe_status cuda_fail(cudaError_t e, const char* where);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace moe

#define REQUIRE_PTR(p, align)                                                          \
  do {                                                                                  \
    if (!(p)) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", #p);                       \
    if (!aligned((p), (align)))                                                         \
      return fail(MOE_ERR_INVALID_ARG, "%s not %d-byte aligned", #p, (int)(align));     \
  } while (0)
