// wgrad.hip — launches of the scale and bias gradients (wgrad.hpp). Compiled
// once per bit width (QP_BITS).
#include <algorithm>

#include "wgrad.hpp"

namespace qp {

namespace {

template <int BITS, int DT>
hipError_t run(const WgradArgs& a, const GradPlan& p, hipStream_t st)
{
    const int64_t tiles = ((a.N + WG_BN - 1) / WG_BN) * ((a.K + WG_BK - 1) / WG_BK);
    hipLaunchKernelGGL((wgrad_f32_kernel<BITS, DT>), dim3((unsigned)tiles, (unsigned)p.splits, (unsigned)a.nmat),
                       dim3(256), 0, st, a, p);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    if (p.splits > 1) {
        const int64_t count = a.N * (a.K / a.gs);
        const int64_t blocks = std::min<int64_t>((2 * count + 255) / 256, 4096);
        for (int mat = 0; mat < a.nmat; ++mat) {
            hipLaunchKernelGGL((wgrad_finish_kernel<DT>), dim3((unsigned)blocks), dim3(256), 0, st,
                               a.partial + (int64_t)mat * 2 * count, p.splits, 2 * count * a.nmat, count,
                               a.dscales[mat], a.dbiases[mat]);
            if (hipError_t e = hipGetLastError(); e != hipSuccess)
                return e;
        }
    }
    return hipSuccess;
}

} // namespace

hipError_t QP_CAT(launch_wgrad_b, QP_BITS)(const WgradArgs& a, const GradPlan& p, hipStream_t st)
{
    switch (a.dt) {
    case DT_F32: return run<QP_BITS, DT_F32>(a, p, st);
    case DT_F16: return run<QP_BITS, DT_F16>(a, p, st);
    case DT_BF16: return run<QP_BITS, DT_BF16>(a, p, st);
    }
    return hipErrorInvalidValue;
}

#if QP_BITS == 4
GradPlan wgrad_plan(int64_t m, int64_t n, int64_t k, int nmat, int, int gs, int)
{
    const int64_t tiles = nmat * ((n + WG_BN - 1) / WG_BN) * ((k + WG_BK - 1) / WG_BK);
    const int64_t steps = (m + WG_M - 1) / WG_M;
    int64_t splits = std::clamp<int64_t>(std::min((512 + tiles - 1) / std::max<int64_t>(tiles, 1), steps / 8), 1, 64);
    GradPlan p{};
    p.tile = 0;
    p.per_split = std::max<int64_t>((steps + splits - 1) / splits, 1);
    p.splits = (int)std::max<int64_t>((steps + p.per_split - 1) / p.per_split, 1);
    p.partial_bytes = p.splits > 1 ? (size_t)p.splits * (size_t)nmat * 2 * (size_t)n * (size_t)(k / gs) * 4 : 0;
    return p;
}
#endif

} // namespace qp
