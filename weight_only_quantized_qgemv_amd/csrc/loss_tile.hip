// loss_tile.hip — launches of the loss's tile kernel (loss_tile.hpp). Compiled once
// per bit width (QP_BITS).
#include <algorithm>

#include "loss_tile.hpp"

namespace qp {

namespace {

template <int DT, int FM, int WMW, bool G32>
hipError_t run(LossTileArgs a, hipStream_t st)
{
    constexpr int LDS = losstile::lds_bytes<QP_BITS, FM, WMW>();
    static_assert(LDS <= 160 * 1024, "LDS budget");
    const void* kern = reinterpret_cast<const void*>(&losstile::loss_tile_kernel<QP_BITS, DT, FM, WMW, G32>);
    static std::atomic<uint64_t> lds{0};   // per instantiation
    if (hipError_t e = allow_lds(lds, kern, LDS); e != hipSuccess)
        return e;
    constexpr int BM = 32 * FM * WMW;
    const int64_t tiles_m = (a.M + BM - 1) / BM, tiles = tiles_m * ((a.N + LOSS_BN - 1) / LOSS_BN);
    a.tiles_m = (int)tiles_m;
    a.tiles = (int)tiles;
    a.per_xcd = (int)((tiles + 7) / 8);
    if (!grid_fits((int64_t)a.per_xcd * 8, 256 * WMW))
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((losstile::loss_tile_kernel<QP_BITS, DT, FM, WMW, G32>), dim3((unsigned)a.per_xcd * 8),
                       dim3(256 * WMW), LDS, st, a);
    return hipGetLastError();
}

template <int DT, bool G32>
hipError_t by_rows(const LossTileArgs& a, hipStream_t st)
{
    if (a.M <= 32) return run<DT, 1, 1, G32>(a, st);
    if (a.M <= 64) return run<DT, 2, 1, G32>(a, st);
    if (a.M <= 128) return run<DT, 4, 1, G32>(a, st);
    return run<DT, 4, 2, G32>(a, st);
}

template <int DT> hipError_t prep_x(const LossTileArgs& a, const void* x, hipStream_t st)
{
    const int units = (a.xn - 2 * a.gp) / 32;
    const int64_t waves = (int64_t)a.M * ((units + 63) / 64), blocks = (waves + 3) / 4;
    if (!grid_fits(blocks, 256))
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((losstile::loss_prep_x_kernel<QP_BITS, DT>), dim3((unsigned)blocks), dim3(256), 0, st,
                       static_cast<const uint16_t*>(x), (int64_t)a.M, a.K, a.gs, a.xn, a.gp,
                       static_cast<uint16_t*>(const_cast<void*>(a.xp)));
    return hipGetLastError();
}

} // namespace

hipError_t QP_CAT(launch_loss_prep_x_b, QP_BITS)(int dt, const LossTileArgs& a, const void* x, hipStream_t st)
{
    return dt == DT_F16 ? prep_x<DT_F16>(a, x, st) : prep_x<DT_BF16>(a, x, st);
}

hipError_t QP_CAT(launch_loss_tile_b, QP_BITS)(int dt, LossTileArgs a, hipStream_t st)
{
    if (dt == DT_F16)
        return a.gs == 32 ? by_rows<DT_F16, true>(a, st) : by_rows<DT_F16, false>(a, st);
    return a.gs == 32 ? by_rows<DT_BF16, true>(a, st) : by_rows<DT_BF16, false>(a, st);
}

} // namespace qp
