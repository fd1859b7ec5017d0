// train_driver.cpp — calls the C-ABI entry points of the operators that train and score a
// model (api_train.cpp) with argument errors, valid shapes and sizes at the ends of int64,
// against the stub launchers below. Built with the host side under AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_sanitize_train.py; no GPU is touched.
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../include/qpack.h"
#include "../../weight_only_quantized_qgemv_amd/csrc/train_ops.hpp"

static int launches = 0, failures = 0;

namespace qp {
hipError_t launch_norm(const NormArgs&, hipStream_t) { return ++launches, hipSuccess; }
size_t norm_grad_workspace_bytes(int64_t, int64_t d, int64_t) { return (size_t)d * 12; }
hipError_t launch_norm_grad(const NormGradArgs&, hipStream_t) { return ++launches, hipSuccess; }
size_t loss_workspace_bytes(int64_t m, int64_t, int64_t, int, int, int) { return (size_t)m * 16; }
hipError_t launch_loss(const LossArgs&, hipStream_t) { return ++launches, hipSuccess; }
size_t loss_grad_workspace_bytes(int64_t m, int64_t, int64_t, int, int, int) { return (size_t)m * 16; }
hipError_t launch_loss_grad(const LossGradArgs&, hipStream_t) { return ++launches, hipSuccess; }
} // namespace qp

static void expect(const char* what, qp_status got, qp_status want, int n, int want_n)
{
    if (got != want || n != want_n || (want != QP_OK && std::strlen(qpack_last_error()) == 0)) {
        std::fprintf(stderr, "FAIL %s: status %d, want %d, %d launches, want %d (%s)\n", what, (int)got, (int)want, n,
                     want_n, qpack_last_error());
        ++failures;
    }
}
#define RUN(what, call, want, n)                        \
    do {                                                \
        const int l0 = launches;                        \
        const qp_status s = (call);                     \
        expect(what, s, want, launches - l0, n);        \
    } while (0)

int main()
{
    void* A = reinterpret_cast<void*>(0x10000);   // stand-in addresses, never dereferenced
    void* ODD = reinterpret_cast<void*>(0x10001);
    const uint32_t* W = static_cast<const uint32_t*>(A);
    const int32_t* I = static_cast<const int32_t*>(A);
    float* F = static_cast<float*>(A);
    const size_t ALL = ~(size_t)0;
    const int64_t ends[] = {INT64_MIN, -1, 0, 1, 64, INT32_MAX, (int64_t)INT32_MAX + 1, INT64_MAX / 64, INT64_MAX};

    auto loss = [&](int64_t m, int64_t k, int64_t v, int bits, const void* x, size_t nws) {
        return qcross_entropy(x, QP_BF16, m, k, I, W, A, A, QP_BF16, v, bits, 64, F, F, A, nws, nullptr);
    };
    RUN("qcross_entropy", loss(2, 128, 100, 4, A, ALL), QP_OK, 1);
    RUN("qcross_entropy bits", loss(2, 128, 100, 5, A, ALL), QP_ERR_UNSUPPORTED, 0);
    RUN("qcross_entropy k", loss(2, 100, 100, 4, A, ALL), QP_ERR_SHAPE, 0);
    RUN("qcross_entropy x", loss(2, 128, 100, 4, ODD, ALL), QP_ERR_ALIGN, 0);
    RUN("qcross_entropy ws", loss(2, 128, 100, 4, A, 3), QP_ERR_WORKSPACE, 0);
    RUN("qcross_entropy no rows", loss(0, 128, 100, 4, nullptr, ALL), QP_OK, 0);
    RUN("qcross_entropy no vocabulary", loss(2, 128, 0, 4, nullptr, ALL), QP_OK, 1);
    auto back = [&](int64_t m, int64_t k, int64_t v, void* dx, void* ds, void* db) {
        return qcross_entropy_backward(A, QP_F16, m, k, I, F, F, W, A, A, QP_F16, v, 6, 32, dx, ds, db, A, ALL, nullptr);
    };
    RUN("qcross_entropy_backward", back(2, 64, 100, A, A, A), QP_OK, 1);
    RUN("qcross_entropy_backward nothing", back(2, 64, 100, nullptr, nullptr, nullptr), QP_OK, 0);
    RUN("qcross_entropy_backward half", back(2, 64, 100, A, A, nullptr), QP_ERR_INVALID_ARG, 0);
    RUN("qcross_entropy_backward no rows", back(0, 64, 100, A, A, A), QP_OK, 1);

    auto norm = [&](int64_t m, int64_t d, int64_t g, const void* y, void* out) {
        return qblock_norm(A, QP_F32, m, d, y, QP_F16, A, y, y, g, 1.0f, 0.0f, 1e-6f, A, out, nullptr);
    };
    RUN("qblock_norm", norm(4, 100, 2, A, A), QP_OK, 1);
    RUN("qblock_norm without y", norm(4, 100, 2, nullptr, A), QP_OK, 1);
    RUN("qblock_norm gates", norm(4, 100, 3, A, A), QP_ERR_SHAPE, 0);
    RUN("qblock_norm out", norm(4, 100, 2, A, nullptr), QP_ERR_INVALID_ARG, 0);
    auto norm_back = [&](int64_t m, int64_t d, int64_t g, void* dy, void* ws) {
        return qblock_norm_backward(A, A, QP_BF16, m, d, A, A, QP_BF16, A, A, A, g, 1.0f, 1.0f, 1e-6f, A, dy, A, A, A,
                                    ws, ALL, nullptr);
    };
    RUN("qblock_norm_backward", norm_back(4, 100, 4, A, A), QP_OK, 1);
    RUN("qblock_norm_backward dy", norm_back(4, 100, 4, ODD, A), QP_ERR_ALIGN, 0);
    RUN("qblock_norm_backward ws", norm_back(4, 100, 4, A, nullptr), QP_ERR_INVALID_ARG, 0);

    // Sizes at the ends: a status, and no overflow on the way to it.
    for (int64_t a : ends)
        for (int64_t b : ends)
            for (int64_t c : ends) {
                (void)loss(a, b, c, 4, A, ALL);
                (void)back(a, b, c, A, A, A);
                (void)norm(a, b, c, A, A);
                (void)norm_back(a, b, c, A, A);
                (void)qcross_entropy_workspace_bytes(a, b, c, 4, 64, QP_BF16);
                (void)qcross_entropy_backward_workspace_bytes(a, b, c, 8, 32, QP_F32);
                (void)qblock_norm_backward_workspace_bytes(a, b, c);
            }
    if (failures == 0)
        std::puts("all calls clean");
    return failures != 0;
}
