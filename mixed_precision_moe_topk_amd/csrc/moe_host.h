// Host helpers shared by the files that implement the C ABI (defined in
// moe_api.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/moe.h"

namespace moe {

// Records a failure of the calling thread for moe_last_error.
moe_status set_error(moe_status st, const char* msg);
moe_status set_errorf(moe_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the calling thread's message.
moe_status set_ok();
// A launch's status; with MOE_SYNC_CHECK=1 synchronises and names the kernel.
moe_status check_hip(hipError_t e, const char* what, hipStream_t st);
// MOE_ERR_UNSUPPORTED unless the current device is a gfx950.
moe_status check_gfx950();
// Dims, num_tokens and top_k in the ranges of the run calls.
moe_status check_layer(const moe_dims* dims, int64_t num_tokens, int32_t top_k);

inline bool is_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace moe

#define MOE_RETURN_IF(expr)           \
  do {                                \
    moe_status _s = (expr);           \
    if (_s != MOE_OK) return _s;      \
  } while (0)
