// api_model.cpp — the C ABI of the operators around the quantized products
// (declared in include/qpack.h): argument validation on the host, then the
// launches on the caller's stream. Every check runs before any HIP call, so
// the error paths work on a machine without a GPU. The rules on bits, group
// size, packing and types are those of the products (api.cpp).
#include "../../include/qpack.h"
#include "api_checks.hpp"
#include "model_ops.hpp"

using namespace qp::api;

namespace {

bool act_ok(int a) { return a == QP_SILU || a == QP_GELU_TANH; }

// Types, sizes and layout of the gated block's calls.
qp_status check_ffn(const char* what, int dt, int sdt, int64_t m, int64_t d, int64_t f, int32_t bits, int32_t gs,
                    int act)
{
    if (m < 0 || d < 0 || f < 0)
        return fail(QP_ERR_INVALID_ARG, "%s: negative size (m=%lld, d_model=%lld, d_ff=%lld)", what, (long long)m,
                    (long long)d, (long long)f);
    if (!dtype_ok(dt) || !dtype_ok(sdt))
        return fail(QP_ERR_INVALID_ARG, "%s: unknown dtype (x=%d, scales=%d)", what, dt, sdt);
    if (!act_ok(act))
        return fail(QP_ERR_UNSUPPORTED, "%s: activation %d not supported (0 SiLU, 1 GELU with tanh)", what, act);
    if (qp_status s = check_layout(d, bits, gs); s != QP_OK)
        return s;
    if (qp_status s = check_layout(f, bits, gs); s != QP_OK)
        return s;
    if (dt != sdt)
        return fail(QP_ERR_DTYPE_MISMATCH, "%s: input dtype %d must match scales dtype %d", what, dt, sdt);
    if (m > kMaxDim || d > kMaxDim || f > kMaxDim || !mul_ok(m, d) || !mul_ok(m, f) || !mul_ok(d, f) ||
        !mul_ok(m * f, 64) || !mul_ok(m * d, 64) || !mul_ok(d * f, 64))
        return fail(QP_ERR_INVALID_ARG, "%s: size too large", what);
    return QP_OK;
}

} // namespace

extern "C" {

size_t qffn_workspace_bytes(int64_t m, int64_t d_model, int64_t d_ff, qp_dtype dtype)
{
    if (m < 0 || d_model < 0 || d_ff < 0 || !dtype_ok(dtype) || !mul_ok(m, d_ff) || !mul_ok(m * d_ff, 64) ||
        !mul_ok(m, d_model) || !mul_ok(m * d_model, 64))
        return 0;
    return qp::ffn_workspace_bytes(m, d_model, d_ff, (int)dtype);
}

qp_status qffn(const void* x, qp_dtype x_dtype, int64_t m, int64_t d_model, int64_t d_ff, const uint32_t* gate_wq,
               const void* gate_scales, const void* gate_biases, const uint32_t* up_wq, const void* up_scales,
               const void* up_biases, const uint32_t* down_wq, const void* down_scales, const void* down_biases,
               qp_dtype sb_dtype, int32_t bits, int32_t group_size, qp_act act, void* saved, void* y,
               void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    const char* what = "qffn";
    if (qp_status s = check_ffn(what, x_dtype, sb_dtype, m, d_model, d_ff, bits, group_size, act); s != QP_OK)
        return s;
    if (m == 0)
        return ok();
    const size_t es = esize(x_dtype);
    if (!aligned(saved, es))
        return fail(QP_ERR_ALIGN, "%s: saved not aligned to its element size", what);
    if (d_model > 0) {
        if (qp_status s = check_tensor(what, "y", y, es); s != QP_OK)
            return s;
    }
    if (d_model > 0 && d_ff > 0) {
        if (qp_status s = check_tensor(what, "x", x, es); s != QP_OK)
            return s;
        if (qp_status s = check_weight(what, "gate", gate_wq, gate_scales, gate_biases, es); s != QP_OK)
            return s;
        if (qp_status s = check_weight(what, "up", up_wq, up_scales, up_biases, es); s != QP_OK)
            return s;
        if (qp_status s = check_weight(what, "down", down_wq, down_scales, down_biases, es); s != QP_OK)
            return s;
    }
    if (qp_status s = check_workspace(what, workspace, workspace_bytes,
                                      qp::ffn_workspace_bytes(m, d_model, d_ff, (int)x_dtype)); s != QP_OK)
        return s;
    qp::FfnArgs a{};
    a.x = x; a.dt = (int)x_dtype; a.act = (int)act;
    a.M = m; a.D = d_model; a.F = d_ff;
    a.gate = {gate_wq, gate_scales, gate_biases};
    a.up = {up_wq, up_scales, up_biases};
    a.down = {down_wq, down_scales, down_biases};
    a.bits = bits; a.gs = group_size;
    if (saved) {
        a.saved[0] = saved;
        a.saved[1] = static_cast<char*>(saved) + (size_t)m * (size_t)d_ff * es;
    }
    a.y = y; a.workspace = workspace;
    return hip_result(qp::launch_ffn(a, stream), what);
}

size_t qffn_backward_workspace_bytes(int64_t m, int64_t d_model, int64_t d_ff, int32_t bits, int32_t group_size,
                                     qp_dtype dtype)
{
    if (check_ffn("qffn_backward", dtype, dtype, m, d_model, d_ff, bits, group_size, QP_SILU) != QP_OK)
        return 0;
    return qp::ffn_grad_workspace_bytes(m, d_model, d_ff, group_size, (int)dtype);
}

qp_status qffn_backward(const void* x, const void* dy, const void* saved, qp_dtype x_dtype, int64_t m,
                        int64_t d_model, int64_t d_ff, const uint32_t* gate_wq, const void* gate_scales,
                        const void* gate_biases, const uint32_t* up_wq, const void* up_scales,
                        const void* up_biases, const uint32_t* down_wq, const void* down_scales,
                        const void* down_biases, qp_dtype sb_dtype, int32_t bits, int32_t group_size, qp_act act,
                        void* dx, void* dgate_scales, void* dgate_biases, void* dup_scales, void* dup_biases,
                        void* ddown_scales, void* ddown_biases, void* workspace, size_t workspace_bytes,
                        hipStream_t stream)
{
    const char* what = "qffn_backward";
    if (qp_status s = check_ffn(what, x_dtype, sb_dtype, m, d_model, d_ff, bits, group_size, act); s != QP_OK)
        return s;
    const size_t es = esize(x_dtype);
    if (qp_status s = check_grads(what, "gate", dgate_scales, dgate_biases, es); s != QP_OK)
        return s;
    if (qp_status s = check_grads(what, "up", dup_scales, dup_biases, es); s != QP_OK)
        return s;
    if (qp_status s = check_grads(what, "down", ddown_scales, ddown_biases, es); s != QP_OK)
        return s;
    if (!aligned(dx, es))
        return fail(QP_ERR_ALIGN, "%s: dx not aligned to its element size", what);
    if (!dx && !dgate_scales && !dup_scales && !ddown_scales)
        return ok();
    if (m > 0 && d_model > 0 && d_ff > 0) {
        if (dgate_scales || dup_scales)
            if (qp_status s = check_tensor(what, "x", x, es); s != QP_OK)
                return s;
        if (qp_status s = check_tensor(what, "dy", dy, es); s != QP_OK)
            return s;
        if (qp_status s = check_tensor(what, "saved", saved, es); s != QP_OK)
            return s;
        if (qp_status s = check_weight(what, "gate", gate_wq, gate_scales, gate_biases, es); s != QP_OK)
            return s;
        if (qp_status s = check_weight(what, "up", up_wq, up_scales, up_biases, es); s != QP_OK)
            return s;
        if (qp_status s = check_weight(what, "down", down_wq, down_scales, down_biases, es); s != QP_OK)
            return s;
        if (qp_status s = check_workspace(what, workspace, workspace_bytes,
                                          qp::ffn_grad_workspace_bytes(m, d_model, d_ff, group_size,
                                                                       (int)x_dtype)); s != QP_OK)
            return s;
    }
    qp::FfnGradArgs a{};
    a.x = x; a.dy = dy; a.saved = saved; a.dt = (int)x_dtype; a.act = (int)act;
    a.M = m; a.D = d_model; a.F = d_ff;
    a.gate = {gate_wq, gate_scales, gate_biases};
    a.up = {up_wq, up_scales, up_biases};
    a.down = {down_wq, down_scales, down_biases};
    a.bits = bits; a.gs = group_size;
    a.dx = dx;
    a.dgate[0] = dgate_scales; a.dgate[1] = dgate_biases;
    a.dup[0] = dup_scales; a.dup[1] = dup_biases;
    a.ddown[0] = ddown_scales; a.ddown[1] = ddown_biases;
    a.workspace = workspace;
    return hip_result(qp::launch_ffn_grad(a, stream), what);
}

static qp_status check_linear(const char* what, int dt, int sdt, int64_t m, int64_t k, int64_t n, int32_t bits,
                              int32_t gs)
{
    if (m < 0 || k < 0 || n < 0)
        return fail(QP_ERR_INVALID_ARG, "%s: negative size (m=%lld, k=%lld, n=%lld)", what, (long long)m,
                    (long long)k, (long long)n);
    if (!dtype_ok(dt) || !dtype_ok(sdt))
        return fail(QP_ERR_INVALID_ARG, "%s: unknown dtype (x=%d, scales=%d)", what, dt, sdt);
    if (qp_status s = check_layout(k, bits, gs); s != QP_OK)
        return s;
    if (dt != sdt)
        return fail(QP_ERR_DTYPE_MISMATCH, "%s: input dtype %d must match scales dtype %d", what, dt, sdt);
    if (m > kMaxDim || k > kMaxDim || n > kMaxDim || !mul_ok(m, k) || !mul_ok(m, n) || !mul_ok(n, k) ||
        !mul_ok(m * k, 64) || !mul_ok(m * n, 64) || !mul_ok(n * k, 64))
        return fail(QP_ERR_INVALID_ARG, "%s: size too large", what);
    return QP_OK;
}

size_t qmatmul_backward_workspace_bytes(int64_t m, int64_t k, int64_t n, int32_t bits, int32_t group_size,
                                        qp_dtype dtype)
{
    if (check_linear("qmatmul_backward", dtype, dtype, m, k, n, bits, group_size) != QP_OK)
        return 0;
    return qp::linear_grad_workspace_bytes(m, k, n, group_size, (int)dtype);
}

qp_status qmatmul_backward(const void* x, const void* dy, qp_dtype x_dtype, int64_t m, int64_t k,
                           const uint32_t* wq, const void* scales, const void* biases, qp_dtype sb_dtype, int64_t n,
                           int32_t bits, int32_t group_size, void* dx, void* dscales, void* dbiases,
                           void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    const char* what = "qmatmul_backward";
    if (qp_status s = check_linear(what, x_dtype, sb_dtype, m, k, n, bits, group_size); s != QP_OK)
        return s;
    const size_t es = esize(x_dtype);
    if (qp_status s = check_grads(what, "weight", dscales, dbiases, es); s != QP_OK)
        return s;
    if (!aligned(dx, es))
        return fail(QP_ERR_ALIGN, "%s: dx not aligned to its element size", what);
    if (!dx && !dscales)
        return ok();
    if (m > 0 && k > 0 && n > 0) {
        if (dscales)
            if (qp_status s = check_tensor(what, "x", x, es); s != QP_OK)
                return s;
        if (qp_status s = check_tensor(what, "dy", dy, es); s != QP_OK)
            return s;
        if (qp_status s = check_weight(what, "the", wq, scales, biases, es); s != QP_OK)
            return s;
        if (qp_status s = check_workspace(what, workspace, workspace_bytes,
                                          qp::linear_grad_workspace_bytes(m, k, n, group_size,
                                                                          (int)x_dtype)); s != QP_OK)
            return s;
    }
    qp::LinearGradArgs a{};
    a.x = x; a.dy = dy; a.dt = (int)x_dtype;
    a.M = m; a.K = k; a.N = n;
    a.w = {wq, scales, biases};
    a.bits = bits; a.gs = group_size;
    a.dx = dx; a.dscales = dscales; a.dbiases = dbiases;
    a.workspace = workspace;
    return hip_result(qp::launch_linear_grad(a, stream), what);
}

static qp_status check_table(const char* what, int dt, int64_t t, int64_t v, int64_t k, int32_t bits, int32_t gs)
{
    if (t < 0 || v < 0 || k < 0)
        return fail(QP_ERR_INVALID_ARG, "%s: negative size (tokens=%lld, rows=%lld, k=%lld)", what, (long long)t,
                    (long long)v, (long long)k);
    if (!dtype_ok(dt))
        return fail(QP_ERR_INVALID_ARG, "%s: unknown dtype %d", what, dt);
    if (qp_status s = check_layout(k, bits, gs); s != QP_OK)
        return s;
    if (t > kMaxDim / 4 || v > kMaxDim - 2 || k > kMaxDim || !mul_ok(t, k) || !mul_ok(v, k) || !mul_ok(t * k, 64) ||
        !mul_ok(v * k, 64))
        return fail(QP_ERR_INVALID_ARG, "%s: size too large", what);
    return QP_OK;
}

qp_status qembedding(const int32_t* ids, int64_t n_tokens, const uint32_t* wq, const void* scales,
                     const void* biases, qp_dtype sb_dtype, int64_t n_rows, int64_t k, int32_t bits,
                     int32_t group_size, float factor, void* out, hipStream_t stream)
{
    const char* what = "qembedding";
    if (qp_status s = check_table(what, sb_dtype, n_tokens, n_rows, k, bits, group_size); s != QP_OK)
        return s;
    if (n_tokens == 0 || k == 0)
        return ok();
    const size_t es = esize(sb_dtype);
    if (qp_status s = check_tensor(what, "out", out, es); s != QP_OK)
        return s;
    if (qp_status s = check_tensor(what, "ids", ids, 4); s != QP_OK)
        return s;
    if (n_rows > 0)
        if (qp_status s = check_weight(what, "table", wq, scales, biases, es); s != QP_OK)
            return s;
    qp::EmbedArgs a{};
    a.ids = ids; a.T = n_tokens; a.V = n_rows; a.K = k;
    a.table = {wq, scales, biases};
    a.dt = (int)sb_dtype; a.bits = bits; a.gs = group_size;
    a.factor = factor; a.out = out;
    return hip_result(qp::launch_embedding(a, stream), what);
}

size_t qembedding_backward_workspace_bytes(int64_t n_tokens, int64_t k, int32_t bits, int32_t group_size)
{
    if (check_table("qembedding_backward", QP_F32, n_tokens, 0, k, bits, group_size) != QP_OK)
        return 0;
    return qp::embedding_grad_workspace_bytes(n_tokens, k, group_size);
}

qp_status qembedding_backward(const int32_t* ids, int64_t n_tokens, const void* dout, qp_dtype dtype,
                              const uint32_t* wq, int64_t n_rows, int64_t k, int32_t bits, int32_t group_size,
                              float factor, void* dscales, void* dbiases, void* workspace, size_t workspace_bytes,
                              hipStream_t stream)
{
    const char* what = "qembedding_backward";
    if (qp_status s = check_table(what, dtype, n_tokens, n_rows, k, bits, group_size); s != QP_OK)
        return s;
    if (n_rows == 0 || k == 0)
        return ok();
    const size_t es = esize(dtype);
    if (qp_status s = check_tensor(what, "dscales", dscales, es); s != QP_OK)
        return s;
    if (qp_status s = check_tensor(what, "dbiases", dbiases, es); s != QP_OK)
        return s;
    if (n_tokens > 0) {
        if (qp_status s = check_tensor(what, "ids", ids, 4); s != QP_OK)
            return s;
        if (qp_status s = check_tensor(what, "dout", dout, es); s != QP_OK)
            return s;
        if (qp_status s = check_tensor(what, "wq", wq, 4); s != QP_OK)
            return s;
        if (qp_status s = check_workspace(what, workspace, workspace_bytes,
                                          qp::embedding_grad_workspace_bytes(n_tokens, k, group_size)); s != QP_OK)
            return s;
    }
    qp::EmbedGradArgs a{};
    a.ids = ids; a.dout = dout; a.wq = wq;
    a.T = n_tokens; a.V = n_rows; a.K = k;
    a.dt = (int)dtype; a.bits = bits; a.gs = group_size;
    a.factor = factor;
    a.dscales = dscales; a.dbiases = dbiases;
    a.workspace = workspace;
    return hip_result(qp::launch_embedding_grad(a, stream), what);
}

qp_status qlogits_adjust(const void* logits, qp_dtype dtype, int64_t rows, int64_t vocab, int64_t in_stride,
                         const int32_t* history, int64_t history_len, const int32_t* history_offsets,
                         const int32_t* prompt_lens, const float* repetition, const float* frequency,
                         const float* presence, const int32_t* bias_ids, const float* bias_values, int64_t bias_len,
                         const int32_t* bias_offsets, const uint32_t* mask, int64_t mask_stride, void* out,
                         int64_t out_stride, hipStream_t stream)
{
    const char* what = "qlogits_adjust";
    if (rows < 0 || vocab < 0 || history_len < 0 || bias_len < 0)
        return fail(QP_ERR_INVALID_ARG, "%s: negative size (rows=%lld, vocab=%lld, history=%lld, bias=%lld)", what,
                    (long long)rows, (long long)vocab, (long long)history_len, (long long)bias_len);
    if (!dtype_ok(dtype))
        return fail(QP_ERR_INVALID_ARG, "%s: unknown dtype %d", what, (int)dtype);
    if (rows > kMaxDim || vocab > kMaxDim || history_len > kMaxDim || bias_len > kMaxDim || in_stride > kMaxDim ||
        out_stride > kMaxDim || mask_stride > kMaxDim || !mul_ok(rows, (vocab + 4095) / 4096) ||
        rows * ((vocab + 4095) / 4096) > kMaxDim / 4)
        return fail(QP_ERR_INVALID_ARG, "%s: size too large", what);
    if (rows > 1 && (in_stride < vocab || out_stride < vocab))
        return fail(QP_ERR_SHAPE, "%s: row stride (%lld in, %lld out) below vocab=%lld", what, (long long)in_stride,
                    (long long)out_stride, (long long)vocab);
    if (mask && mask_stride != 0 && mask_stride < (vocab + 31) / 32)
        return fail(QP_ERR_SHAPE, "%s: mask stride %lld below %lld words (or 0, one mask for all rows)", what,
                    (long long)mask_stride, (long long)((vocab + 31) / 32));
    if (rows == 0 || vocab == 0)
        return ok();
    const size_t es = esize(dtype);
    if (qp_status s = check_tensor(what, "logits", logits, es); s != QP_OK)
        return s;
    if (qp_status s = check_tensor(what, "out", out, es); s != QP_OK)
        return s;
    if ((repetition || frequency || presence) && !history_offsets)
        return fail(QP_ERR_INVALID_ARG, "%s: penalties need the rows' tokens (history, history_offsets)", what);
    if (history_offsets && history_len > 0 && !history)
        return fail(QP_ERR_INVALID_ARG, "%s: null history", what);
    if (bias_offsets && bias_len > 0 && (!bias_ids || !bias_values))
        return fail(QP_ERR_INVALID_ARG, "%s: null bias ids or values", what);
    if ((history && !history_offsets) || (bias_ids && !bias_offsets))
        return fail(QP_ERR_INVALID_ARG, "%s: tokens without their rows' offsets", what);
    if (!aligned(history, 4) || !aligned(history_offsets, 4) || !aligned(prompt_lens, 4) || !aligned(repetition, 4) ||
        !aligned(frequency, 4) || !aligned(presence, 4) || !aligned(bias_ids, 4) || !aligned(bias_values, 4) ||
        !aligned(bias_offsets, 4) || !aligned(mask, 4))
        return fail(QP_ERR_ALIGN, "%s: pointer not aligned to its element size", what);
    qp::LogitsArgs a{};
    a.logits = logits; a.dt = (int)dtype;
    a.rows = rows; a.vocab = vocab; a.in_stride = in_stride;
    const bool pen = history_len > 0 && (repetition || frequency || presence);
    a.history = pen ? history : nullptr; a.history_len = history_len; a.offsets = history_offsets;
    a.prompt_lens = prompt_lens;
    a.repetition = repetition; a.frequency = frequency; a.presence = presence;
    a.bias_ids = bias_len > 0 ? bias_ids : nullptr; a.bias_values = bias_values; a.bias_len = bias_len;
    a.bias_offsets = bias_offsets;
    a.mask = mask; a.mask_stride = mask_stride;
    a.out = out; a.out_stride = out_stride;
    return hip_result(qp::launch_logits_adjust(a, stream), what);
}

} // extern "C"
