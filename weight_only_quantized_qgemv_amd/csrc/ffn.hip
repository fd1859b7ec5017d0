// ffn.hip — the dense gated feed-forward block over packed weights:
//   h = act(x Wg^T) * (x Wu^T),   y = h Wd^T
// (the block of qgemv_moe_ffn, ferrum-kernels src/stacked_expert.rs, with one
// set of weights for every row).
#include <algorithm>

#include "act.hpp"
#include "common.hpp"
#include "model_ops.hpp"
#include "xgrad.hpp"

namespace qp {

namespace {

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// h[i] = act(g[i]) u[i], rounded once; h may be g's own memory.
template <int DT>
__global__ __launch_bounds__(256) void ffn_gate_kernel(const void* g, const void* u, int act, int64_t n, void* h)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        store_elem<DT>(h, i, act_f32(act, load_elem<DT>(g, i)) * load_elem<DT>(u, i));
}

hipError_t gate(const FfnArgs& a, const void* g, const void* u, void* h, hipStream_t st)
{
    const int64_t n = a.M * a.F;
    const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, 16384);
    switch (a.dt) {
    case DT_F32:
        hipLaunchKernelGGL((ffn_gate_kernel<DT_F32>), dim3(blocks), dim3(256), 0, st, g, u, a.act, n, h);
        break;
    case DT_F16:
        hipLaunchKernelGGL((ffn_gate_kernel<DT_F16>), dim3(blocks), dim3(256), 0, st, g, u, a.act, n, h);
        break;
    case DT_BF16:
        hipLaunchKernelGGL((ffn_gate_kernel<DT_BF16>), dim3(blocks), dim3(256), 0, st, g, u, a.act, n, h);
        break;
    default:
        return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

// y = x W^T on qmatmul's kernels. The tile kernel reads activations in 16-byte
// pieces; other alignments take the decode kernels, which test for it.
hipError_t product(const FfnArgs& a, const void* x, int64_t k, const QWeight& w, int64_t n, void* y, hipStream_t st)
{
    if (k == 0)
        return launch_fill_zero(y, a.dt, a.M * n, st);
    GemvArgs g{x, a.dt, a.M, k, n, w.wq, w.scales, w.biases, a.bits, a.gs, y};
    if (a.M <= 16 || a.dt == DT_F32 || !aligned16(x))
        return launch_qgemv(g, st);
    return launch_qgemm(g, st);
}

hipError_t gate_up(const GateUpArgs& a, hipStream_t st, bool* done)
{
    switch (a.bits) {
    case 2: return launch_gate_up_b2(a, st, done);
    case 3: return launch_gate_up_b3(a, st, done);
    case 4: return launch_gate_up_b4(a, st, done);
    case 6: return launch_gate_up_b6(a, st, done);
    case 8: return launch_gate_up_b8(a, st, done);
    }
    return hipErrorInvalidValue;
}

size_t elem_size(int dt) { return dt == DT_F32 ? 4 : 2; }
size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

} // namespace

// h, and the up projection's product where the two products are separate
// launches and the caller does not keep them.
size_t ffn_workspace_bytes(int64_t m, int64_t f, int dt)
{
    return 2 * up16((size_t)m * (size_t)f * elem_size(dt));
}

hipError_t launch_ffn(const FfnArgs& a, hipStream_t st)
{
    const size_t hb = up16((size_t)a.M * (size_t)a.F * elem_size(a.dt));
    char* const h = static_cast<char*>(a.workspace);
    char* const g = a.saved != nullptr ? static_cast<char*>(a.saved) : h;
    char* const u = a.saved != nullptr ? g + (size_t)a.M * (size_t)a.F * elem_size(a.dt) : h + hb;
    bool done = false;
    if (a.F > 0 && a.D > 0) {
        GateUpArgs k{a.x, a.dt, a.act, a.M, a.D, a.F, a.gate, a.up, a.bits, a.gs, h, a.saved};
        if (hipError_t e = gate_up(k, st, &done); e != hipSuccess)
            return e;
    }
    if (a.F > 0 && !done) {
        if (hipError_t e = product(a, a.x, a.D, a.gate, a.F, g, st); e != hipSuccess)
            return e;
        if (hipError_t e = product(a, a.x, a.D, a.up, a.F, u, st); e != hipSuccess)
            return e;
        if (hipError_t e = gate(a, g, u, h, st); e != hipSuccess)
            return e;
    }
    if (a.D == 0)
        return hipSuccess;
    return product(a, h, a.F, a.down, a.D, a.y, st);
}

} // namespace qp
