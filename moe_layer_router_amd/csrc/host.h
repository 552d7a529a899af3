// What the host parts of the library share: the error text behind
// moe_last_error, argument checks and the device check.  Defined in
// kernels.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_layer.h"

namespace moe {

// Records the calling thread's error text and returns s.
moe_status fail(moe_status s, const char* fmt, ...);

// Non-NULL (when required) and 16-byte aligned.
moe_status check_ptr(const void* p, const char* name, bool required = true);

struct DevInfo {
  int checked = 0, ok = 0, cus = 0;
};
// The current device: MOE_ERR_UNSUPPORTED unless it is a gfx950.
moe_status device_info(DevInfo* out);

// Whether two buffers share bytes.
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a && b && a0 < b0 + nb && b0 < a0 + na;
}

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

#define TRY(expr)                       \
  do {                                  \
    moe_status _s = (expr);             \
    if (_s != MOE_OK) return _s;        \
  } while (0)

#define HIP_TRY(expr)                                                                    \
  do {                                                                                   \
    hipError_t _e = (expr);                                                              \
    if (_e != hipSuccess) return fail(MOE_ERR_HIP, "%s: %s", #expr, hipGetErrorString(_e)); \
  } while (0)

// Dynamic LDS above the default limit has to be allowed per kernel.
template <typename K>
moe_status set_lds_limit(K kernel, int bytes) {
  if (bytes > 64 * 1024) HIP_TRY(hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes));
  return MOE_OK;
}

}  // namespace moe
