// grad.hip — the backward passes, put together from the input-gradient and
// weight-gradient products (xgrad.hpp, wgrad.hpp).
//   linear layer y = x W^T:  dx = dy W;  dW = dy^T x
//   gated block:             dh = dy Wd, closed into dg, du and h;
//                            dx = dg Wg + du Wu;
//                            dWg = dg^T x, dWu = du^T x, dWd = dy^T h
// and of each dW only the sums that belong to the scales and biases.
#include <algorithm>

#include "common.hpp"
#include "model_ops.hpp"

namespace qp {

namespace {

size_t elem_size(int dt) { return dt == DT_F32 ? 4 : 2; }
size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

hipError_t xgrad(const XgradArgs& a, const GradPlan& p, hipStream_t st)
{
    switch (a.bits) {
    case 2: return launch_xgrad_b2(a, p, st);
    case 3: return launch_xgrad_b3(a, p, st);
    case 4: return launch_xgrad_b4(a, p, st);
    case 6: return launch_xgrad_b6(a, p, st);
    case 8: return launch_xgrad_b8(a, p, st);
    }
    return hipErrorInvalidValue;
}

hipError_t wgrad(const WgradArgs& a, const GradPlan& p, hipStream_t st)
{
    switch (a.bits) {
    case 2: return launch_wgrad_b2(a, p, st);
    case 3: return launch_wgrad_b3(a, p, st);
    case 4: return launch_wgrad_b4(a, p, st);
    case 6: return launch_wgrad_b6(a, p, st);
    case 8: return launch_wgrad_b8(a, p, st);
    }
    return hipErrorInvalidValue;
}

// Zeros for a weight's gradients (no rows to sum over).
hipError_t zero_grads(void* ds, void* db, int dt, int64_t count, hipStream_t st)
{
    if (ds == nullptr || count == 0)
        return hipSuccess;
    if (hipError_t e = launch_fill_zero(ds, dt, count, st); e != hipSuccess)
        return e;
    return launch_fill_zero(db, dt, count, st);
}

} // namespace

size_t linear_grad_workspace_bytes(int64_t m, int64_t k, int64_t n, int bits, int gs, int dt)
{
    if (m == 0 || k == 0 || n == 0)
        return 0;
    return std::max(xgrad_plan(m, n, k, 1, bits, dt).partial_bytes,
                    wgrad_plan(m, n, k, 1, bits, gs, dt).partial_bytes);
}

hipError_t launch_linear_grad(const LinearGradArgs& a, hipStream_t st)
{
    if (a.dx != nullptr && a.M * a.K > 0) {
        if (a.N == 0) {
            if (hipError_t e = launch_fill_zero(a.dx, a.dt, a.M * a.K, st); e != hipSuccess)
                return e;
        } else {
            XgradArgs x{};
            x.dy[0] = x.dy[1] = a.dy;
            x.dy_stride = a.N;
            x.w[0] = x.w[1] = a.w;
            x.nmat = 1;
            x.dt = a.dt;
            x.M = a.M; x.N = a.N; x.K = a.K;
            x.bits = a.bits; x.gs = a.gs;
            x.out = a.dx;
            x.partial = static_cast<float*>(a.workspace);
            if (hipError_t e = xgrad(x, xgrad_plan(a.M, a.N, a.K, 1, a.bits, a.dt), st); e != hipSuccess)
                return e;
        }
    }
    if (a.dscales == nullptr || a.N * a.K == 0)
        return hipSuccess;
    if (a.M == 0)
        return zero_grads(a.dscales, a.dbiases, a.dt, a.N * (a.K / a.gs), st);
    WgradArgs w{};
    w.x = a.x;
    w.dy[0] = w.dy[1] = a.dy;
    w.dy_stride = a.N;
    w.wq[0] = w.wq[1] = a.w.wq;
    w.nmat = 1;
    w.dt = a.dt;
    w.M = a.M; w.N = a.N; w.K = a.K;
    w.bits = a.bits; w.gs = a.gs;
    w.dscales[0] = a.dscales;
    w.dbiases[0] = a.dbiases;
    w.partial = static_cast<float*>(a.workspace);
    return wgrad(w, wgrad_plan(a.M, a.N, a.K, 1, a.bits, a.gs, a.dt), st);
}

// dg, du and h, then the partial sums of one product at a time.
size_t ffn_grad_workspace_bytes(int64_t m, int64_t d, int64_t f, int bits, int gs, int dt)
{
    if (m == 0 || d == 0 || f == 0)
        return 0;
    size_t part = xgrad_plan(m, d, f, 1, bits, dt).partial_bytes;
    part = std::max(part, xgrad_plan(m, f, d, 2, bits, dt).partial_bytes);
    part = std::max(part, wgrad_plan(m, f, d, 2, bits, gs, dt).partial_bytes);
    part = std::max(part, wgrad_plan(m, f, d, 1, bits, gs, dt).partial_bytes);
    part = std::max(part, wgrad_plan(m, d, f, 1, bits, gs, dt).partial_bytes);
    return 3 * up16((size_t)m * (size_t)f * elem_size(dt)) + part;
}

hipError_t launch_ffn_grad(const FfnGradArgs& a, hipStream_t st)
{
    const int64_t M = a.M, D = a.D, F = a.F;
    if (M == 0 || D == 0 || F == 0) {
        if (a.dx != nullptr && M * D > 0)
            if (hipError_t e = launch_fill_zero(a.dx, a.dt, M * D, st); e != hipSuccess)
                return e;
        const int64_t count = D * F / a.gs;
        if (hipError_t e = zero_grads(a.dgate[0], a.dgate[1], a.dt, count, st); e != hipSuccess)
            return e;
        if (hipError_t e = zero_grads(a.dup[0], a.dup[1], a.dt, count, st); e != hipSuccess)
            return e;
        return zero_grads(a.ddown[0], a.ddown[1], a.dt, count, st);
    }
    const size_t mf = (size_t)M * (size_t)F * elem_size(a.dt), step = up16(mf);
    char* const dg = static_cast<char*>(a.workspace);
    char* const du = dg + step;
    char* const h = du + step;
    float* const partial = reinterpret_cast<float*>(h + step);

    XgradArgs x{};
    x.dt = a.dt; x.act = a.act; x.M = M; x.bits = a.bits; x.gs = a.gs;
    x.partial = partial;
    x.dy[0] = x.dy[1] = a.dy;
    x.dy_stride = D;
    x.w[0] = x.w[1] = a.down;
    x.nmat = 1;
    x.N = D; x.K = F;
    x.g = a.saved;
    x.u = static_cast<const char*>(a.saved) + mf;
    x.dg = dg; x.du = du;
    x.h = a.ddown[0] != nullptr ? h : nullptr;
    if (hipError_t e = xgrad(x, xgrad_plan(M, D, F, 1, a.bits, a.dt), st); e != hipSuccess)
        return e;
    if (a.dx != nullptr) {
        x.g = x.u = nullptr;
        x.dy[0] = dg; x.dy[1] = du;
        x.dy_stride = F;
        x.w[0] = a.gate; x.w[1] = a.up;
        x.nmat = 2;
        x.N = F; x.K = D;
        x.out = a.dx;
        if (hipError_t e = xgrad(x, xgrad_plan(M, F, D, 2, a.bits, a.dt), st); e != hipSuccess)
            return e;
    }
    WgradArgs w{};
    w.dt = a.dt; w.M = M; w.bits = a.bits; w.gs = a.gs;
    w.partial = partial;
    w.x = a.x;
    w.N = F; w.K = D;
    w.dy_stride = F;
    w.nmat = 0;
    auto add = [&](const char* dy, const QWeight& q, void* const (&grads)[2]) {
        if (grads[0] == nullptr)
            return;
        w.dy[w.nmat] = dy;
        w.wq[w.nmat] = q.wq;
        w.dscales[w.nmat] = grads[0];
        w.dbiases[w.nmat] = grads[1];
        ++w.nmat;
    };
    add(dg, a.gate, a.dgate);
    add(du, a.up, a.dup);
    if (w.nmat > 0)
        if (hipError_t e = wgrad(w, wgrad_plan(M, F, D, w.nmat, a.bits, a.gs, a.dt), st); e != hipSuccess)
            return e;
    if (a.ddown[0] == nullptr)
        return hipSuccess;
    w.x = h;
    w.N = D; w.K = F;
    w.dy_stride = D;
    w.nmat = 0;
    add(static_cast<const char*>(a.dy), a.down, a.ddown);
    return wgrad(w, wgrad_plan(M, D, F, 1, a.bits, a.gs, a.dt), st);
}

} // namespace qp
