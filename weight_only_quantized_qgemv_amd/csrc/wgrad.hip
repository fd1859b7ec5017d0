// wgrad.hip — launches of the scale and bias gradients (wgrad.hpp). Compiled
// once per bit width (QP_BITS), and once more with QP_SCALED for calls with a factor.
#include <algorithm>

#include "gradtile.hpp"
#include "wgrad.hpp"

namespace qp {

namespace {

#ifdef QP_SCALED
constexpr bool SCALED = true;
#else
constexpr bool SCALED = false;
#endif

template <int BITS, int DT, int BT>
hipError_t run_tile(const WgradArgs& a, const GradPlan& p, hipStream_t st)
{
    constexpr int LDS = gradtile::wgrad_lds<BT, BT>();
    static_assert(LDS <= 160 * 1024, "LDS budget");
    const void* kern = reinterpret_cast<const void*>(&gradtile::wgrad_tile_kernel<BITS, DT, BT, BT, SCALED>);
    static std::atomic<uint64_t> lds{0};   // per instantiation
    if (hipError_t e = allow_lds(lds, kern, LDS); e != hipSuccess)
        return e;
    const int64_t tiles_k = (a.K + BT - 1) / BT, tiles = (a.N + BT - 1) / BT * tiles_k;
    const int per_xcd = (int)((tiles * a.nmat + 7) / 8);
    if (!grid_fits((int64_t)per_xcd * 8, 2 * BT))
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((gradtile::wgrad_tile_kernel<BITS, DT, BT, BT, SCALED>),
                       dim3((unsigned)per_xcd * 8, (unsigned)p.splits), dim3(2 * BT), LDS, st, a, p, (int)tiles_k, (int)tiles,
                       per_xcd);
    return hipGetLastError();
}

template <int BITS, int DT>
hipError_t run_wide(const WgradArgs& a, hipStream_t st)
{
    constexpr int BT = 256, LDS = gradtile::wgrad_lds<BT, BT>();
    const void* kern = reinterpret_cast<const void*>(&gradtile::wgrad_wide_kernel<BITS, DT, SCALED>);
    static std::atomic<uint64_t> lds{0};   // per instantiation
    if (hipError_t e = allow_lds(lds, kern, LDS); e != hipSuccess)
        return e;
    int cus = 0;
    if (hipError_t e = device_cu_count(&cus); e != hipSuccess)
        return e;
    const int64_t tiles_n = (a.N + BT - 1) / BT, tiles_k = (a.K + BT - 1) / BT;
    const int64_t items = tiles_n * tiles_k * a.nmat;
    const int64_t blocks = std::min<int64_t>((items + 7) / 8 * 8, std::max(cus / 8 * 8, 8));
    hipLaunchKernelGGL((gradtile::wgrad_wide_kernel<BITS, DT, SCALED>), dim3((unsigned)blocks), dim3(256), LDS, st, a,
                       (int)tiles_n, (int)tiles_k);
    return hipGetLastError();
}

template <int BITS, int DT>
hipError_t run(const WgradArgs& a, const GradPlan& p, hipStream_t st)
{
    hipError_t e = hipErrorInvalidValue;
    if (p.tile == 0) {
        const int64_t tiles = ((a.N + WG_BN - 1) / WG_BN) * ((a.K + WG_BK - 1) / WG_BK);
        if (!grid_fits(tiles, 256))
            return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL((wgrad_f32_kernel<BITS, DT, SCALED>), dim3((unsigned)tiles, (unsigned)p.splits, (unsigned)a.nmat),
                           dim3(256), 0, st, a, p);
        e = hipGetLastError();
    } else if constexpr (DT != DT_F32) {
        e = p.tile == 1 ? run_wide<BITS, DT>(a, st) : run_tile<BITS, DT, 128>(a, p, st);
    }
    if (e != hipSuccess)
        return e;
    if (p.splits > 1) {
        const int64_t count = a.N * (a.K / a.gs);
        const int64_t blocks = std::min<int64_t>((2 * count + 255) / 256, 4096);
        for (int mat = 0; mat < a.nmat; ++mat) {
            hipLaunchKernelGGL((wgrad_finish_kernel<DT, SCALED>), dim3((unsigned)blocks), dim3(256), 0, st,
                               a.partial + (int64_t)mat * 2 * count, p.splits, 2 * count * a.nmat, count,
                               a.dscales[mat], a.dbiases[mat], a.scale);
            if (hipError_t e = hipGetLastError(); e != hipSuccess)
                return e;
        }
    }
    return hipSuccess;
}

} // namespace

#ifdef QP_SCALED
hipError_t QP_CAT(launch_wgrad_scaled_b, QP_BITS)(const WgradArgs& a, const GradPlan& p, hipStream_t st)
#else
hipError_t QP_CAT(launch_wgrad_b, QP_BITS)(const WgradArgs& a, const GradPlan& p, hipStream_t st)
#endif
{
    switch (a.dt) {
#ifndef QP_SCALED   // (16-bit operands have factors)
    case DT_F32: return run<QP_BITS, DT_F32>(a, p, st);
#endif
    case DT_F16: return run<QP_BITS, DT_F16>(a, p, st);
    case DT_BF16: return run<QP_BITS, DT_BF16>(a, p, st);
    }
    return hipErrorInvalidValue;
}

#if QP_BITS == 4 && !defined(QP_SCALED)
// The wide kernel where its 256 x 256 tiles reach every CU: 2048 rows of a 14336
// x 4096 weight 227 us, tiles of 128 304; 1024 rows of 4096 x 2048 (128 tiles)
// 27.2 and 25.4. So too where a second round is all but empty (4352 x 4096, 272
// tiles: 2048 rows 107.5 and 107.3, 256 rows 28.8 and 25.9; 320 tiles 107.5 and
// 113.1, 27.9 and 25.6). The others in pieces of the rows, at least four steps
// each, until there are two blocks a CU.
GradPlan wgrad_plan(int64_t m, int64_t n, int64_t k, int nmat, int gs, bool tile_kernels)
{
    GradPlan p{};
    auto count = [&](int64_t b) { return nmat * ((n + b - 1) / b) * ((k + b - 1) / b); };
    p.tile = !tile_kernels ? 0 : count(256) >= 256 ? 1 : 2;
    const int64_t step = p.tile == 0 ? WG_M : gradtile::STEP, steps = (m + step - 1) / step;
    const int64_t splits = p.tile == 1
        ? 1 : std::clamp<int64_t>(std::min(512 / std::max<int64_t>(count(128), 1), steps / 4), 1, 64);
    p.per_split = std::max<int64_t>((steps + splits - 1) / splits, 1);
    p.splits = (int)std::max<int64_t>((steps + p.per_split - 1) / p.per_split, 1);
    p.partial_bytes = p.splits > 1 ? (size_t)p.splits * (size_t)nmat * 2 * (size_t)n * (size_t)(k / gs) * 4 : 0;
    return p;
}
#endif

} // namespace qp
