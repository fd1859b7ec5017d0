// xgrad.hip — launches of the input-gradient products (xgrad.hpp). Compiled
// once per bit width (QP_BITS).
#include <algorithm>

#include "xgrad.hpp"

namespace qp {

namespace {

template <int DT>
hipError_t finish(const XgradArgs& a, int splits, hipStream_t st)
{
    const int64_t blocks = std::min<int64_t>((a.M * a.K + 255) / 256, 16384);
    hipLaunchKernelGGL((xgrad_finish_kernel<DT>), dim3((unsigned)blocks), dim3(256), 0, st, a, splits);
    return hipGetLastError();
}

template <int BITS, int DT>
hipError_t run(const XgradArgs& a, const GradPlan& p, hipStream_t st)
{
    const int64_t tiles = ((a.M + XG_BM - 1) / XG_BM) * ((a.K + XG_BK - 1) / XG_BK);
    hipLaunchKernelGGL((xgrad_f32_kernel<BITS, DT>), dim3((unsigned)tiles, (unsigned)p.splits), dim3(256), 0, st,
                       a, p);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    return p.splits > 1 ? finish<DT>(a, p.splits, st) : hipSuccess;
}

} // namespace

hipError_t QP_CAT(launch_xgrad_b, QP_BITS)(const XgradArgs& a, const GradPlan& p, hipStream_t st)
{
    switch (a.dt) {
    case DT_F32: return run<QP_BITS, DT_F32>(a, p, st);
    case DT_F16: return run<QP_BITS, DT_F16>(a, p, st);
    case DT_BF16: return run<QP_BITS, DT_BF16>(a, p, st);
    }
    return hipErrorInvalidValue;
}

#if QP_BITS == 4
GradPlan xgrad_plan(int64_t m, int64_t n, int64_t k, int nmat, int, int)
{
    // Pieces of the contraction until there are about two blocks a CU, none
    // shorter than eight steps.
    const int64_t tiles = ((m + XG_BM - 1) / XG_BM) * ((k + XG_BK - 1) / XG_BK);
    const int64_t steps = nmat * ((n + XG_N - 1) / XG_N);
    int64_t splits = std::clamp<int64_t>(std::min((512 + tiles - 1) / std::max<int64_t>(tiles, 1), steps / 8), 1, 64);
    GradPlan p{};
    p.tile = 0;
    p.per_split = std::max<int64_t>((steps + splits - 1) / splits, 1);
    p.splits = (int)std::max<int64_t>((steps + p.per_split - 1) / p.per_split, 1);
    p.partial_bytes = p.splits > 1 ? (size_t)p.splits * (size_t)m * (size_t)k * 4 : 0;
    return p;
}
#endif

} // namespace qp
