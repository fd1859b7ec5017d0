// api_checks.hpp — the host checks and the error record that the C ABI files
// share (defined in api.cpp).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/qpack.h"

namespace qp {
namespace api {

// Records the message as the calling thread's last error and returns s.
qp_status fail(qp_status s, const char* fmt, ...);
// Clears it and returns QP_OK.
qp_status ok();
qp_status hip_result(hipError_t e, const char* what);

inline bool dtype_ok(int d) { return d == QP_F32 || d == QP_F16 || d == QP_BF16; }
inline size_t esize(int d) { return d == QP_F32 ? 4 : 2; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// a * b without int64 overflow (both non-negative).
inline bool mul_ok(int64_t a, int64_t b) { return a == 0 || b <= INT64_MAX / a; }

// Checks shared by every call: bits, group size, K divisibility.
qp_status check_layout(int64_t k, int32_t bits, int32_t gs);

} // namespace api
} // namespace qp
