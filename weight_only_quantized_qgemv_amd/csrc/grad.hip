// grad.hip — the backward passes, put together from the input-gradient and
// weight-gradient products (xgrad.hpp, wgrad.hpp).
//   linear layer y = x W^T:  dx = dy W;  dW = dy^T x
//   gated block:             dh = dy Wd, closed into dg, du and h;
//                            dx = dg Wg + du Wu;
//                            dWg = dg^T x, dWu = du^T x, dWd = dy^T h
// and of each dW only the sums that belong to the scales and biases. dg, du and h
// are rounded once to the activations' type, because they are the operands of the
// next products on 16-bit instructions: in bf16 the gradients are 0.0032 of their
// size off 64 bits where one rounding of the result gives 0.0017. In fp32 nothing
// is rounded.
#include <algorithm>

#include "act.hpp"
#include "common.hpp"
#include "model_ops.hpp"
#include "xgrad.hpp"

namespace qp {

namespace {

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

int64_t up8(int64_t n) { return (n + 7) & ~(int64_t)7; }

// Whether the tile kernels' 32-bit offsets reach a tile's rows: rows of at
// most 2^20 elements.
bool tile_sizes(int64_t n, int64_t k, int dt) { return dt != DT_F32 && n <= (1 << 20) && k <= (1 << 20); }

// The tile kernel rounds each weight to the activations' type. Over fewer than
// 64 rows (one step, the shortest contraction of the forward tiles too) those
// roundings, up to 2^-8 of a bfloat16 weight, do not average out: the fp32
// kernel takes such a product.
bool averages(int64_t n) { return n >= 64; }

// The larger of the two kernels' partial sums: which one runs depends on the
// pointers too.
size_t xgrad_bytes(int64_t m, int64_t n, int64_t k, int nmat)
{
    return std::max(xgrad_plan(m, n, k, nmat, false).partial_bytes, xgrad_plan(m, n, k, nmat, true).partial_bytes);
}
size_t wgrad_bytes(int64_t m, int64_t n, int64_t k, int nmat, int gs)
{
    return std::max(wgrad_plan(m, n, k, nmat, gs, false).partial_bytes, wgrad_plan(m, n, k, nmat, gs, true).partial_bytes);
}

// Rows of n 16-bit elements copied to rows of up8(n), zeros between.
__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t* __restrict__ in, int64_t m, int64_t n,
                                                       int64_t n8, uint16_t* __restrict__ out)
{
    const int64_t octets = m * (n8 / 8);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < octets; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / (n8 / 8), c = 8 * (i - r * (n8 / 8));
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = c + j < n ? in[r * n + c + j] : 0u;
        reinterpret_cast<u32x4_t*>(out)[i] = u32x4_t{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
    }
}

// The tile kernels read 16-bit rows in 16-byte pieces: rows p [m, n] as they lie
// where they are such, else in a copy at `to`, zeros between; *stride their distance.
hipError_t pieces_of_rows(const void*& p, int64_t m, int64_t n, char* to, int64_t* stride, hipStream_t st)
{
    *stride = n;
    if (n % 8 == 0 && aligned16(p))
        return hipSuccess;
    *stride = up8(n);
    const unsigned blocks = (unsigned)std::min<int64_t>((m * (*stride / 8) + 255) / 256, 16384);
    hipLaunchKernelGGL(pad_rows_kernel, dim3(blocks), dim3(256), 0, st, static_cast<const uint16_t*>(p), m, n, *stride,
                       reinterpret_cast<uint16_t*>(to));
    p = to;
    return hipGetLastError();
}
size_t piece_bytes(int64_t m, int64_t n) { return up16((size_t)m * (size_t)up8(n) * 2); }

// h[i] = act(g[i]) u[i] as the close of dh forms it, for a call that asks for the
// down projection's gradients alone: dh is not needed there.
template <int DT>
__global__ __launch_bounds__(256) void ffn_hidden_kernel(const void* g, const void* u, int act, int64_t n, void* h)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        float a, da;
        act_grad_f32(act, load_elem<DT>(g, i), a, da);
        store_elem<DT>(h, i, a * load_elem<DT>(u, i));
    }
}
hipError_t hidden(int dt, const void* g, const void* u, int act, int64_t n, void* h, hipStream_t st)
{
    const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, 16384);
    switch (dt) {
    case DT_F32: hipLaunchKernelGGL(ffn_hidden_kernel<DT_F32>, dim3(blocks), dim3(256), 0, st, g, u, act, n, h); break;
    case DT_F16: hipLaunchKernelGGL(ffn_hidden_kernel<DT_F16>, dim3(blocks), dim3(256), 0, st, g, u, act, n, h); break;
    default: hipLaunchKernelGGL(ffn_hidden_kernel<DT_BF16>, dim3(blocks), dim3(256), 0, st, g, u, act, n, h);
    }
    return hipGetLastError();
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

// Room for copies of dy and x, then the partial sums of one product at a time.
size_t linear_grad_workspace_bytes(int64_t m, int64_t k, int64_t n, int gs, int dt)
{
    if (m == 0 || k == 0 || n == 0)
        return 0;
    return (tile_sizes(n, k, dt) ? piece_bytes(m, n) + piece_bytes(m, k) : 0) +
           std::max(xgrad_bytes(m, n, k, 1), wgrad_bytes(m, n, k, 1, gs));
}

hipError_t launch_linear_grad(const LinearGradArgs& a, hipStream_t st)
{
    const int64_t M = a.M, N = a.N, K = a.K;
    if (M == 0 || N == 0 || K == 0) {
        if (a.dx != nullptr && M * K > 0)
            if (hipError_t e = launch_fill_zero(a.dx, a.dt, M * K, st); e != hipSuccess)
                return e;
        return zero_grads(a.dscales, a.dbiases, a.dt, N * (K / a.gs), st);
    }
    const void *dy = a.dy, *xs = a.x;
    int64_t stride = N, xstride = K;
    const bool tiles = tile_sizes(N, K, a.dt);
    char* room = static_cast<char*>(a.workspace);
    if (tiles) {
        if (hipError_t e = pieces_of_rows(dy, M, N, room, &stride, st); e != hipSuccess)
            return e;
        room += piece_bytes(M, N);
        if (a.dscales != nullptr)   // x is not read otherwise
            if (hipError_t e = pieces_of_rows(xs, M, K, room, &xstride, st); e != hipSuccess)
                return e;
        room += piece_bytes(M, K);
    }
    float* const partial = reinterpret_cast<float*>(room);
    if (a.dx != nullptr) {
        XgradArgs x{};
        x.dy[0] = x.dy[1] = dy;
        x.dy_stride = stride;
        x.w[0] = x.w[1] = a.w;
        x.nmat = 1;
        x.dt = a.dt;
        x.M = M; x.N = N; x.K = K;
        x.bits = a.bits; x.gs = a.gs;
        x.out = a.dx;
        x.partial = partial;
        if (hipError_t e = xgrad(x, xgrad_plan(M, N, K, 1, tiles && averages(N)), st); e != hipSuccess)
            return e;
    }
    if (a.dscales == nullptr)
        return hipSuccess;
    WgradArgs w{};
    w.x = xs;
    w.dy[0] = w.dy[1] = dy;
    w.dy_stride = stride;
    w.wq[0] = w.wq[1] = a.w.wq;
    w.nmat = 1;
    w.dt = a.dt;
    w.M = M; w.N = N; w.K = K;
    w.bits = a.bits; w.gs = a.gs;
    w.dscales[0] = a.dscales;
    w.dbiases[0] = a.dbiases;
    w.partial = partial;
    return wgrad(w, wgrad_plan(M, N, K, 1, a.gs, tiles), st);
}

// dg, du and h, room for copies of dy and x, then the partial sums of one product
// at a time.
size_t ffn_grad_workspace_bytes(int64_t m, int64_t d, int64_t f, int gs, int dt)
{
    if (m == 0 || d == 0 || f == 0)
        return 0;
    size_t part = std::max(xgrad_bytes(m, d, f, 1), xgrad_bytes(m, f, d, 2));
    part = std::max(part, std::max(wgrad_bytes(m, f, d, 2, gs), wgrad_bytes(m, f, d, 1, gs)));
    part = std::max(part, wgrad_bytes(m, d, f, 1, gs));
    return 3 * up16((size_t)m * (size_t)f * elem_size(dt)) +
           (tile_sizes(d, f, dt) ? 2 * piece_bytes(m, d) : 0) + part;
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
    char* room = h + step;

    const bool tiles = tile_sizes(D, F, a.dt);
    const void *dy = a.dy, *xs = a.x;
    if (tiles) {
        int64_t stride = D;   // whole pieces: it stays
        if (hipError_t e = pieces_of_rows(dy, M, D, room, &stride, st); e != hipSuccess)
            return e;
        room += piece_bytes(M, D);
        if (a.dgate[0] != nullptr || a.dup[0] != nullptr)   // x is not read otherwise
            if (hipError_t e = pieces_of_rows(xs, M, D, room, &stride, st); e != hipSuccess)
                return e;
        room += piece_bytes(M, D);
    }
    float* const partial = reinterpret_cast<float*>(room);

    XgradArgs x{};
    x.dt = a.dt; x.act = a.act; x.M = M; x.bits = a.bits; x.gs = a.gs;
    x.partial = partial;
    x.dy[0] = x.dy[1] = dy;
    x.dy_stride = D;
    x.w[0] = x.w[1] = a.down;
    x.nmat = 1;
    x.N = D; x.K = F;
    x.g = a.saved;
    x.u = static_cast<const char*>(a.saved) + mf;
    x.dg = dg; x.du = du;
    x.h = a.ddown[0] != nullptr ? h : nullptr;
    const bool down_only = a.dx == nullptr && a.dgate[0] == nullptr && a.dup[0] == nullptr;
    if (hipError_t e = down_only ? hidden(a.dt, x.g, x.u, a.act, M * F, h, st)
                                 : xgrad(x, xgrad_plan(M, D, F, 1, tiles && averages(D)), st); e != hipSuccess)
        return e;
    if (a.dx != nullptr) {
        x.g = x.u = nullptr;
        x.dy[0] = dg; x.dy[1] = du;
        x.dy_stride = F;
        x.w[0] = a.gate; x.w[1] = a.up;
        x.nmat = 2;
        x.N = F; x.K = D;
        x.out = a.dx;
        if (hipError_t e = xgrad(x, xgrad_plan(M, F, D, 2, tiles && averages(F)), st); e != hipSuccess)
            return e;
    }
    WgradArgs w{};
    w.dt = a.dt; w.M = M; w.bits = a.bits; w.gs = a.gs;
    w.partial = partial;
    w.x = xs;
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
        if (hipError_t e = wgrad(w, wgrad_plan(M, F, D, w.nmat, a.gs, tiles), st); e != hipSuccess)
            return e;
    if (a.ddown[0] == nullptr)
        return hipSuccess;
    w.x = h;
    w.N = D; w.K = F;
    w.dy_stride = D;
    w.nmat = 0;
    add(static_cast<const char*>(dy), a.down, a.ddown);
    return wgrad(w, wgrad_plan(M, D, F, 1, a.gs, tiles), st);
}

} // namespace qp
