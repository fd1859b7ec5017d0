// model_driver.cpp — calls the C-ABI entry points of the operators around the
// products (api_model.cpp) with argument errors (each must return its status
// and launch nothing), with valid shapes (each must reach its launcher) and
// with sizes at the ends of int64, against the stub launchers below. Built with
// the host side under AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_sanitize_model.py; no GPU is touched.
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../include/qpack.h"
#include "../../weight_only_quantized_qgemv_amd/csrc/model_ops.hpp"

static int launches = 0, failures = 0;

namespace qp {
size_t ffn_workspace_bytes(int64_t m, int64_t, int64_t f, int) { return (size_t)m * (size_t)f * 4; }
hipError_t launch_ffn(const FfnArgs&, hipStream_t) { return ++launches, hipSuccess; }
size_t linear_grad_workspace_bytes(int64_t m, int64_t, int64_t n, int, int) { return (size_t)m * (size_t)n; }
hipError_t launch_linear_grad(const LinearGradArgs&, hipStream_t) { return ++launches, hipSuccess; }
size_t ffn_grad_workspace_bytes(int64_t m, int64_t, int64_t f, int, int) { return (size_t)m * (size_t)f * 6; }
hipError_t launch_ffn_grad(const FfnGradArgs&, hipStream_t) { return ++launches, hipSuccess; }
hipError_t launch_embedding(const EmbedArgs&, hipStream_t) { return ++launches, hipSuccess; }
size_t embedding_grad_workspace_bytes(int64_t t, int64_t, int) { return (size_t)t * 8; }
hipError_t launch_embedding_grad(const EmbedGradArgs&, hipStream_t) { return ++launches, hipSuccess; }
hipError_t launch_logits_adjust(const LogitsArgs&, hipStream_t) { return ++launches, hipSuccess; }
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
    const float* F = static_cast<const float*>(A);
    const size_t ALL = ~(size_t)0;
    const int64_t ends[] = {INT64_MIN, -1, 0, 1, 64, INT32_MAX, (int64_t)INT32_MAX + 1, INT64_MAX / 64, INT64_MAX};

    auto ffn = [&](int64_t m, int64_t d, int64_t f, int bits, int gs, int act, void* y, void* ws, size_t nws) {
        return qffn(A, QP_BF16, m, d, f, W, A, A, W, A, A, W, A, A, QP_BF16, bits, gs, (qp_act)act, nullptr, y, ws,
                    nws, nullptr);
    };
    RUN("qffn", ffn(2, 128, 256, 4, 64, 0, A, A, ALL), QP_OK, 1);
    RUN("qffn bits", ffn(2, 128, 256, 7, 64, 0, A, A, ALL), QP_ERR_UNSUPPORTED, 0);
    RUN("qffn act", ffn(2, 128, 256, 4, 64, 9, A, A, ALL), QP_ERR_UNSUPPORTED, 0);
    RUN("qffn d", ffn(2, 100, 256, 4, 64, 0, A, A, ALL), QP_ERR_SHAPE, 0);
    RUN("qffn y", ffn(2, 128, 256, 4, 64, 0, nullptr, A, ALL), QP_ERR_INVALID_ARG, 0);
    RUN("qffn ws", ffn(2, 128, 256, 4, 64, 0, A, A, 1), QP_ERR_WORKSPACE, 0);
    RUN("qffn odd ws", ffn(2, 128, 256, 4, 64, 0, A, ODD, ALL), QP_ERR_ALIGN, 0);

    auto back = [&](int64_t m, int64_t d, int64_t f, void* dx, void* ds, void* db) {
        return qffn_backward(A, A, A, QP_F32, m, d, f, W, A, A, W, A, A, W, A, A, QP_F32, 4, 64, QP_GELU_TANH, dx,
                             ds, db, ds, db, ds, db, A, ALL, nullptr);
    };
    RUN("qffn_backward", back(2, 128, 256, A, A, A), QP_OK, 1);
    RUN("qffn_backward nothing", back(2, 128, 256, nullptr, nullptr, nullptr), QP_OK, 0);
    RUN("qffn_backward half", back(2, 128, 256, A, A, nullptr), QP_ERR_INVALID_ARG, 0);

    auto linear = [&](int64_t m, int64_t k, int64_t n, void* dx, void* ds, size_t nws) {
        return qmatmul_backward(A, A, QP_F16, m, k, W, A, A, QP_F16, n, 3, 32, dx, ds, ds, A, nws, nullptr);
    };
    RUN("qmatmul_backward", linear(5, 64, 7, A, A, ALL), QP_OK, 1);
    RUN("qmatmul_backward ws", linear(5, 64, 7, A, A, 3), QP_ERR_WORKSPACE, 0);
    RUN("qmatmul_backward k", linear(5, 65, 7, A, A, ALL), QP_ERR_SHAPE, 0);
    RUN("qmatmul_backward no rows", linear(0, 64, 7, A, A, ALL), QP_OK, 1);

    auto embed = [&](int64_t t, int64_t v, int64_t k, void* out) {
        return qembedding(I, t, W, A, A, QP_BF16, v, k, 6, 32, 1.0f, out, nullptr);
    };
    RUN("qembedding", embed(3, 9, 64, A), QP_OK, 1);
    RUN("qembedding none", embed(0, 9, 64, nullptr), QP_OK, 0);
    RUN("qembedding odd", embed(3, 9, 64, ODD), QP_ERR_ALIGN, 0);
    auto embed_back = [&](int64_t t, int64_t v, int64_t k, void* ws) {
        return qembedding_backward(I, t, A, QP_BF16, W, v, k, 6, 32, 1.0f, A, A, ws, ALL, nullptr);
    };
    RUN("qembedding_backward", embed_back(3, 9, 64, A), QP_OK, 1);
    RUN("qembedding_backward ws", embed_back(3, 9, 64, nullptr), QP_ERR_INVALID_ARG, 0);

    auto logits = [&](int64_t rows, int64_t v, int64_t stride, int64_t h, const int32_t* off, int64_t ms) {
        return qlogits_adjust(A, QP_F32, rows, v, stride, I, h, off, nullptr, F, nullptr, nullptr, nullptr, nullptr,
                              0, nullptr, W, ms, A, stride, nullptr);
    };
    RUN("qlogits_adjust", logits(2, 100, 100, 5, I, 4), QP_OK, 1);
    RUN("qlogits_adjust offsets", logits(2, 100, 100, 5, nullptr, 4), QP_ERR_INVALID_ARG, 0);
    RUN("qlogits_adjust stride", logits(2, 100, 50, 5, I, 4), QP_ERR_SHAPE, 0);
    RUN("qlogits_adjust mask", logits(2, 100, 100, 5, I, 2), QP_ERR_SHAPE, 0);

    // Sizes at the ends: a status, and no overflow on the way to it.
    for (int64_t a : ends)
        for (int64_t b : ends)
            for (int64_t c : ends) {
                (void)ffn(a, b, c, 4, 64, 0, A, A, ALL);
                (void)back(a, b, c, A, A, A);
                (void)linear(a, b, c, A, A, ALL);
                (void)embed(a, b, c, A);
                (void)embed_back(a, b, c, A);
                (void)logits(a, b, b, c, I, a);
                (void)qffn_workspace_bytes(a, b, c, QP_BF16);
                (void)qffn_backward_workspace_bytes(a, b, c, 4, 64, QP_F16);
                (void)qmatmul_backward_workspace_bytes(a, b, c, 8, 32, QP_F32);
                (void)qembedding_backward_workspace_bytes(a, b, 2, 32);
            }
    if (failures == 0)
        std::puts("all calls clean");
    return failures != 0;
}
