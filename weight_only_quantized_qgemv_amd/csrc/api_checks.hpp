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

// Checks of the operators around the products.

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;   // sizes are below 2^31

// A packed weight of `count` codes: present and aligned.
inline qp_status check_weight(const char* what, const char* name, const void* wq, const void* scales, const void* biases,
                       size_t es)
{
    if (!wq || !scales || !biases)
        return fail(QP_ERR_INVALID_ARG, "%s: null %s weight pointer", what, name);
    if (!aligned(wq, 4) || !aligned(scales, es) || !aligned(biases, es))
        return fail(QP_ERR_ALIGN, "%s: %s weight pointer not aligned", what, name);
    return QP_OK;
}

// A tensor of the activations' type: present and aligned.
inline qp_status check_tensor(const char* what, const char* name, const void* p, size_t es)
{
    if (!p)
        return fail(QP_ERR_INVALID_ARG, "%s: null %s", what, name);
    if (!aligned(p, es))
        return fail(QP_ERR_ALIGN, "%s: %s not aligned to its element size", what, name);
    return QP_OK;
}

// A pair of gradients: both or neither, aligned.
inline qp_status check_grads(const char* what, const char* name, const void* ds, const void* db, size_t es)
{
    if ((ds == nullptr) != (db == nullptr))
        return fail(QP_ERR_INVALID_ARG, "%s: %s gradients need both scales and biases", what, name);
    if (!aligned(ds, es) || !aligned(db, es))
        return fail(QP_ERR_ALIGN, "%s: %s gradients not aligned to their element size", what, name);
    return QP_OK;
}

inline qp_status check_workspace(const char* what, const void* ws, size_t bytes, size_t need)
{
    if (need == 0)
        return QP_OK;
    if (!ws)
        return fail(QP_ERR_INVALID_ARG, "%s: null workspace", what);
    if (bytes < need)
        return fail(QP_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", what, bytes, need);
    if (!aligned(ws, 16))
        return fail(QP_ERR_ALIGN, "%s: workspace not aligned to 16 bytes", what);
    return QP_OK;
}

} // namespace api
} // namespace qp
