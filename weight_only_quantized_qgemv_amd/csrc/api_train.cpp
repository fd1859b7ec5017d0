// api_train.cpp — the C ABI of the operators that train and score a model around
// the packed layers (declared in include/qpack.h): argument validation on the host,
// then the launches on the caller's stream. Every check runs before any HIP call,
// so the error paths work on a machine without a GPU.
#include <math.h>

#include "../../include/qpack.h"
#include "api_checks.hpp"
#include "train_ops.hpp"

using namespace qp::api;

namespace {

// Types, sizes and layout of the loss's calls.
qp_status check_loss(const char* what, int dt, int sdt, int64_t m, int64_t k, int64_t v, int32_t bits, int32_t gs)
{
    if (m < 0 || k < 0 || v < 0)
        return fail(QP_ERR_INVALID_ARG, "%s: negative size (m=%lld, k=%lld, vocab=%lld)", what, (long long)m,
                    (long long)k, (long long)v);
    if (!dtype_ok(dt) || !dtype_ok(sdt))
        return fail(QP_ERR_INVALID_ARG, "%s: unknown dtype (x=%d, scales=%d)", what, dt, sdt);
    if (qp_status s = check_layout(k, bits, gs); s != QP_OK)
        return s;
    if (dt != sdt)
        return fail(QP_ERR_DTYPE_MISMATCH, "%s: input dtype %d must match scales dtype %d", what, dt, sdt);
    if (m > (1 << 20) || k > (1 << 24) || v > kMaxDim || !mul_ok(v, k) || !mul_ok(v * k, 64))
        return fail(QP_ERR_INVALID_ARG, "%s: size too large", what);
    return QP_OK;
}

// Types and sizes of the norms' calls.
qp_status check_norm(const char* what, int sdt, int dt, int64_t m, int64_t d, bool gate, int64_t gates, float factor,
                     float offset, float eps)
{
    if (m < 0 || d < 0)
        return fail(QP_ERR_INVALID_ARG, "%s: negative size (m=%lld, d=%lld)", what, (long long)m, (long long)d);
    if (!dtype_ok(dt) || !dtype_ok(sdt))
        return fail(QP_ERR_INVALID_ARG, "%s: unknown dtype (stream=%d, block=%d)", what, sdt, dt);
    if (sdt != dt && sdt != QP_F32)
        return fail(QP_ERR_DTYPE_MISMATCH, "%s: the stream's dtype %d must be the block's %d, or fp32", what, sdt, dt);
    if (d > qp::kNormMaxWidth)
        return fail(QP_ERR_UNSUPPORTED, "%s: rows of %lld elements (at most %lld)", what, (long long)d,
                    (long long)qp::kNormMaxWidth);
    if (m > qp::kNormMaxRows)
        return fail(QP_ERR_INVALID_ARG, "%s: size too large", what);
    if (gate && (gates < 0 || (gates == 0 ? m != 0 : m % gates != 0)))
        return fail(QP_ERR_SHAPE, "%s: %lld gate rows do not divide %lld rows", what, (long long)gates, (long long)m);
    if (!isfinite(factor) || !isfinite(offset) || !isfinite(eps) || eps < 0.0f)
        return fail(QP_ERR_INVALID_ARG, "%s: factor, offset and eps must be finite, eps not negative", what);
    return QP_OK;
}

// What the call is to do: something, and a post-norm or gate only of a block's output.
qp_status check_parts(const char* what, const void* y, const void* weight, const void* post, const void* gate)
{
    if (!y && !weight)
        return fail(QP_ERR_INVALID_ARG, "%s: neither a block's output nor a weight: nothing to do", what);
    if (!y && (post || gate))
        return fail(QP_ERR_INVALID_ARG, "%s: a post-norm or gate without a block's output", what);
    return QP_OK;
}

// A tensor that may be absent: aligned.
qp_status check_optional(const char* what, const char* name, const void* p, size_t es)
{
    return p != nullptr ? check_tensor(what, name, p, es) : QP_OK;
}

} // namespace

extern "C" {

size_t qcross_entropy_workspace_bytes(int64_t m, int64_t k, int64_t vocab, int32_t bits, int32_t group_size,
                                      qp_dtype dtype)
{
    if (check_loss("qcross_entropy", dtype, dtype, m, k, vocab, bits, group_size) != QP_OK)
        return 0;
    return qp::loss_workspace_bytes(m, k, vocab, bits, group_size, (int)dtype);
}

qp_status qcross_entropy(const void* x, qp_dtype x_dtype, int64_t m, int64_t k, const int32_t* targets,
                         const uint32_t* wq, const void* scales, const void* biases, qp_dtype sb_dtype, int64_t vocab,
                         int32_t bits, int32_t group_size, float* loss, float* lse, void* workspace,
                         size_t workspace_bytes, hipStream_t stream)
{
    const char* what = "qcross_entropy";
    if (qp_status s = check_loss(what, x_dtype, sb_dtype, m, k, vocab, bits, group_size); s != QP_OK)
        return s;
    if (m == 0)
        return ok();
    const size_t es = esize(x_dtype);
    if (qp_status s = check_tensor(what, "targets", targets, 4); s != QP_OK)
        return s;
    if (qp_status s = check_tensor(what, "loss", loss, 4); s != QP_OK)
        return s;
    if (qp_status s = check_tensor(what, "lse", lse, 4); s != QP_OK)
        return s;
    if (k > 0 && vocab > 0) {
        if (qp_status s = check_tensor(what, "x", x, es); s != QP_OK)
            return s;
        if (qp_status s = check_weight(what, "head", wq, scales, biases, es); s != QP_OK)
            return s;
    }
    if (qp_status s = check_workspace(what, workspace, workspace_bytes,
                                      qp::loss_workspace_bytes(m, k, vocab, bits, group_size, (int)x_dtype));
        s != QP_OK)
        return s;
    qp::LossArgs a{};
    a.x = x; a.dt = (int)x_dtype;
    a.M = m; a.K = k; a.V = vocab;
    a.targets = targets;
    a.w = {wq, scales, biases};
    a.bits = bits; a.gs = group_size;
    a.loss = loss; a.lse = lse;
    a.workspace = workspace;
    return hip_result(qp::launch_loss(a, stream), what);
}

size_t qcross_entropy_backward_workspace_bytes(int64_t m, int64_t k, int64_t vocab, int32_t bits, int32_t group_size,
                                               qp_dtype dtype)
{
    if (check_loss("qcross_entropy_backward", dtype, dtype, m, k, vocab, bits, group_size) != QP_OK)
        return 0;
    return qp::loss_grad_workspace_bytes(m, k, vocab, bits, group_size, (int)dtype);
}

qp_status qcross_entropy_backward(const void* x, qp_dtype x_dtype, int64_t m, int64_t k, const int32_t* targets,
                                  const float* lse, const float* dloss, const uint32_t* wq, const void* scales,
                                  const void* biases, qp_dtype sb_dtype, int64_t vocab, int32_t bits,
                                  int32_t group_size, void* dx, void* dscales, void* dbiases, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream)
{
    const char* what = "qcross_entropy_backward";
    if (qp_status s = check_loss(what, x_dtype, sb_dtype, m, k, vocab, bits, group_size); s != QP_OK)
        return s;
    const size_t es = esize(x_dtype);
    if (qp_status s = check_grads(what, "head", dscales, dbiases, es); s != QP_OK)
        return s;
    if (!aligned(dx, es))
        return fail(QP_ERR_ALIGN, "%s: dx not aligned to its element size", what);
    if (!dx && !dscales)
        return ok();
    if (m > 0 && k > 0 && vocab > 0) {
        if (qp_status s = check_tensor(what, "x", x, es); s != QP_OK)
            return s;
        if (qp_status s = check_tensor(what, "targets", targets, 4); s != QP_OK)
            return s;
        if (qp_status s = check_tensor(what, "lse", lse, 4); s != QP_OK)
            return s;
        if (qp_status s = check_tensor(what, "dloss", dloss, 4); s != QP_OK)
            return s;
        if (qp_status s = check_weight(what, "head", wq, scales, biases, es); s != QP_OK)
            return s;
        if (qp_status s = check_workspace(what, workspace, workspace_bytes,
                                          qp::loss_grad_workspace_bytes(m, k, vocab, bits, group_size, (int)x_dtype));
            s != QP_OK)
            return s;
    }
    qp::LossGradArgs a{};
    a.x = x; a.dt = (int)x_dtype;
    a.M = m; a.K = k; a.V = vocab;
    a.targets = targets;
    a.w = {wq, scales, biases};
    a.bits = bits; a.gs = group_size;
    a.lse = lse; a.dloss = dloss;
    a.dx = dx; a.dscales = dscales; a.dbiases = dbiases;
    a.workspace = workspace;
    return hip_result(qp::launch_loss_grad(a, stream), what);
}

qp_status qblock_norm(const void* x, qp_dtype x_dtype, int64_t m, int64_t d, const void* y, qp_dtype dtype,
                      const void* weight, const void* post_weight, const void* gate, int64_t gate_rows, float scale,
                      float offset, float eps, void* stream_out, void* out, hipStream_t stream)
{
    const char* what = "qblock_norm";
    if (qp_status s = check_norm(what, x_dtype, dtype, m, d, gate != nullptr, gate_rows, scale, offset, eps); s != QP_OK)
        return s;
    if (m == 0 || d == 0)
        return ok();
    if (qp_status s = check_parts(what, y, weight, post_weight, gate); s != QP_OK)
        return s;
    const size_t es = esize(dtype), ss = esize(x_dtype);
    if (qp_status s = check_tensor(what, "x", x, ss); s != QP_OK)
        return s;
    if (qp_status s = check_optional(what, "y", y, es); s != QP_OK)
        return s;
    if (qp_status s = check_optional(what, "weight", weight, es); s != QP_OK)
        return s;
    if (qp_status s = check_optional(what, "post_weight", post_weight, es); s != QP_OK)
        return s;
    if (qp_status s = check_optional(what, "gate", gate, es); s != QP_OK)
        return s;
    if (y)
        if (qp_status s = check_tensor(what, "stream_out", stream_out, ss); s != QP_OK)
            return s;
    if (weight)
        if (qp_status s = check_tensor(what, "out", out, es); s != QP_OK)
            return s;
    qp::NormArgs a{};
    a.x = x; a.sdt = (int)x_dtype; a.dt = (int)dtype;
    a.M = m; a.D = d;
    a.y = y; a.post = post_weight; a.weight = weight;
    a.gate = gate; a.gates = gate ? gate_rows : 1;
    a.factor = scale; a.offset = offset; a.eps = eps;
    a.s = stream_out; a.a = out;
    return hip_result(qp::launch_norm(a, stream), what);
}

size_t qblock_norm_backward_workspace_bytes(int64_t m, int64_t d, int64_t gate_rows)
{
    if (check_norm("qblock_norm_backward", QP_F32, QP_F32, m, d, gate_rows != 0, gate_rows, 1.0f, 0.0f, 0.0f) != QP_OK)
        return 0;
    return qp::norm_grad_workspace_bytes(m, d, gate_rows);
}

qp_status qblock_norm_backward(const void* s, const void* ds, qp_dtype s_dtype, int64_t m, int64_t d, const void* da,
                               const void* y, qp_dtype dtype, const void* weight, const void* post_weight,
                               const void* gate, int64_t gate_rows, float scale, float offset, float eps, void* dx,
                               void* dy, void* dweight, void* dpost_weight, void* dgate, void* workspace,
                               size_t workspace_bytes, hipStream_t stream)
{
    const char* what = "qblock_norm_backward";
    if (qp_status e = check_norm(what, s_dtype, dtype, m, d, gate != nullptr, gate_rows, scale, offset, eps);
        e != QP_OK)
        return e;
    if (d == 0)
        return ok();
    if (m > 0)
        if (qp_status e = check_parts(what, y, weight, post_weight, gate); e != QP_OK)
            return e;
    const size_t es = esize(dtype), ss = esize(s_dtype);
    const struct { const char* name; const void* p; bool need; size_t es; } tensors[] = {
        {"weight", weight, false, es}, {"post_weight", post_weight, false, es}, {"gate", gate, false, es},
        {"dweight", dweight, weight != nullptr, es}, {"dpost_weight", dpost_weight, post_weight != nullptr, es},
        {"dgate", dgate, gate != nullptr, es},
        {"s", s, m > 0 && weight != nullptr, ss}, {"da", da, m > 0 && weight != nullptr, es}, {"ds", ds, false, ss},
        {"y", y, false, es}, {"dx", dx, m > 0, ss}, {"dy", dy, m > 0 && y != nullptr, es}};
    for (const auto& t : tensors)
        if (qp_status e = t.need ? check_tensor(what, t.name, t.p, t.es) : check_optional(what, t.name, t.p, t.es);
            e != QP_OK)
            return e;
    if (qp_status e = check_workspace(what, workspace, workspace_bytes,
                                      qp::norm_grad_workspace_bytes(m, d, gate ? gate_rows : 0)); e != QP_OK)
        return e;
    qp::NormGradArgs a{};
    a.s = s; a.da = da; a.ds = ds; a.y = y;
    a.sdt = (int)s_dtype; a.dt = (int)dtype;
    a.M = m; a.D = d;
    a.post = post_weight; a.weight = weight; a.gate = gate;
    a.gates = gate ? gate_rows : 1;
    a.factor = scale; a.offset = offset; a.eps = eps;
    a.dx = dx; a.dy = dy;
    a.dweight = weight ? dweight : nullptr;
    a.dpost = post_weight ? dpost_weight : nullptr;
    a.dgate = gate ? dgate : nullptr;
    a.workspace = workspace;
    return hip_result(qp::launch_norm_grad(a, stream), what);
}

} // extern "C"
