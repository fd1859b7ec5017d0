// xgrad.hip — launches of the input-gradient products (xgrad.hpp). Compiled
// once per bit width (QP_BITS).
#include <algorithm>

#include "gradtile.hpp"
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

template <int BITS, int DT, int BM, int BN, int WMW>
hipError_t run_tile(const XgradArgs& a, const GradPlan& p, hipStream_t st)
{
    constexpr int LDS = gradtile::xgrad_lds<BM, BN>();
    static_assert(LDS <= 160 * 1024, "LDS budget");
    const void* kern = reinterpret_cast<const void*>(&gradtile::xgrad_tile_kernel<BITS, DT, BM, BN, WMW>);
    static bool attr_set = false;   // per instantiation; set before its first launch
    if (!attr_set) {
        if (hipError_t e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, LDS); e != hipSuccess)
            return e;
        attr_set = true;
    }
    const int64_t tiles_k = (a.K + BN - 1) / BN, tiles = (a.M + BM - 1) / BM * tiles_k;
    const int per_xcd = (int)((tiles + 7) / 8);
    hipLaunchKernelGGL((gradtile::xgrad_tile_kernel<BITS, DT, BM, BN, WMW>), dim3((unsigned)per_xcd * 8, (unsigned)p.splits),
                       dim3(2 * BN), LDS, st, a, p, (int)tiles_k, (int)tiles, per_xcd);
    return hipGetLastError();
}

template <int BITS, int DT>
hipError_t run(const XgradArgs& a, const GradPlan& p, hipStream_t st)
{
    hipError_t e = hipErrorInvalidValue;
    if (p.tile == 0) {
        const int64_t tiles = ((a.M + XG_BM - 1) / XG_BM) * ((a.K + XG_BK - 1) / XG_BK);
        hipLaunchKernelGGL((xgrad_f32_kernel<BITS, DT>), dim3((unsigned)tiles, (unsigned)p.splits), dim3(256), 0, st,
                           a, p);
        e = hipGetLastError();
    } else if constexpr (DT != DT_F32) {
        switch (p.tile) {
        case 1: e = run_tile<BITS, DT, 256, 256, 2>(a, p, st); break;
        case 2: e = run_tile<BITS, DT, 128, 128, 2>(a, p, st); break;
        case 3: e = run_tile<BITS, DT, 64, 128, 2>(a, p, st); break;
        }
    }
    if (e != hipSuccess)
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
GradPlan xgrad_plan(int64_t m, int64_t n, int64_t k, int nmat, bool tile_kernels)
{
    // Pieces of the contraction until there are about two blocks a CU, none
    // shorter than four steps (77 rows of a 1024 x 2816 block's backward: 55.7 us
    // at eight, 50.8 at four, 56.9 at two).
    GradPlan p{};
    p.tile = !tile_kernels ? 0 : m > 128 ? 1 : m > 64 ? 2 : 3;
    const int64_t bm = p.tile == 1 ? 256 : p.tile == 3 ? 64 : 128, bn = p.tile == 1 ? 256 : 128;
    const int64_t step = p.tile == 0 ? XG_N : gradtile::STEP, want = p.tile == 1 ? 256 : 512;
    const int64_t tiles = std::max<int64_t>(((m + bm - 1) / bm) * ((k + bn - 1) / bn), 1);
    const int64_t steps = nmat * ((n + step - 1) / step);
    const int64_t splits = std::clamp<int64_t>(std::min(want / tiles, steps / 4), 1, 64);
    p.per_split = std::max<int64_t>((steps + splits - 1) / splits, 1);
    p.splits = (int)std::max<int64_t>((steps + p.per_split - 1) / p.per_split, 1);
    p.partial_bytes = p.splits > 1 ? (size_t)p.splits * (size_t)m * (size_t)k * 4 : 0;
    return p;
}
#endif

} // namespace qp
