// loss_tile.hip — launches of the loss's tile kernel (loss_tile.hpp). Compiled once
// per bit width (QP_BITS).
#include <algorithm>

#include "loss_tile.hpp"

namespace qp {

namespace {

template <int DT, int FM, int WMW, bool G32>
hipError_t run(LossTileArgs a, hipStream_t st)
{
    constexpr int LDS = losstile::lds_bytes<QP_BITS, DT, FM, WMW, G32>();
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

// The rows of a tile, by an estimate of what a step costs, in us: 32 and 64 rows are two
// blocks a CU once there are more tiles than CUs, the others one. Rounds of the GPU count
// half as whole ones, half as tiles (a round's blocks do not end together). Measured,
// 4096 features, 32000 tokens, 4-bit bf16, tiles of 32 / 64 / 128 / 256 rows: 24 rows 37, 48,
// 71, 104 us; 64 rows 39, 49, 72, 106; 100 rows 63, 53, 73, 106; 200 rows 114, 83, 80,
// 112; 500 rows 242, 165, 159, 135; 1000 rows 508, 352, 337, 263. Other widths' and types'
// steps take up to twice as long, in about the same proportion: with 512, 1024 and 4096
// features, 24 to 500 rows, also of 6- and 8-bit fp16 and 3-bit fp32 in groups of 32 (60
// calls), what is taken is the best of the four or within 2% of it, but for 200 rows of 512
// and 1024 features (at most 7%: 8-bit, 512, 33.5 us on 128 rows and 31.4 on 64).
template <int DT, bool G32>
hipError_t by_rows(const LossTileArgs& a, hipStream_t st)
{
    struct Tile {
        int64_t rows, resident;
        double few, step;   // a step's us with a tile a CU or fewer, with all resident
    };
    constexpr Tile kTiles[] = {{32, 512, 0.52, 0.97}, {64, 512, 0.76, 1.33}, {128, 256, 1.2, 1.29}, {256, 256, 2.1, 2.1}};
    const int64_t tiles_n = (a.N + LOSS_BN - 1) / LOSS_BN;
    int64_t rows = 0;
    double best = 0.0;
    for (const Tile& t : kTiles) {
        const int64_t tiles = (a.M + t.rows - 1) / t.rows * tiles_n, rounds = (tiles + t.resident - 1) / t.resident;
        const double us = tiles <= 256 ? t.few : 0.5 * ((double)rounds + (double)tiles / (double)t.resident) * t.step;
        if (rows == 0 || us < best) {
            rows = t.rows;
            best = us;
        }
    }
    switch (rows) {
    case 32: return run<DT, 1, 1, G32>(a, st);
    case 64: return run<DT, 2, 1, G32>(a, st);
    case 128: return run<DT, 4, 1, G32>(a, st);
    }
    return run<DT, 4, 2, G32>(a, st);
}

template <int DT> hipError_t prep(const LossTileArgs& a, const LossPrepArgs& p, hipStream_t st)
{
    const int units = DT == DT_F32 ? a.xn / 96 : (a.xn - 2 * a.gp) / 32;
    const int64_t waves = p.x != nullptr ? (int64_t)a.M * losstile::prep_waves(DT, (units + 63) / 64) : 0, x_blocks = (waves + 3) / 4;
    const int64_t w_blocks = (int64_t)(a.np / 64) * ((a.gp + 63) / 64);
    const int64_t blocks = w_blocks + x_blocks + (p.factor != nullptr ? 1 : 0);
    if (!grid_fits(blocks, 256))
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((losstile::loss_prep_kernel<QP_BITS, DT>), dim3((unsigned)blocks), dim3(256), 0, st, a, p, w_blocks,
                       x_blocks);
    return hipGetLastError();
}

template <int DT> hipError_t tile(const LossTileArgs& a, hipStream_t st)
{
    return a.gs == 32 ? by_rows<DT, true>(a, st) : by_rows<DT, false>(a, st);
}

} // namespace

hipError_t QP_CAT(launch_loss_prep_b, QP_BITS)(int dt, const LossTileArgs& a, const LossPrepArgs& p, hipStream_t st)
{
    return dt == DT_F32 ? prep<DT_F32>(a, p, st) : dt == DT_F16 ? prep<DT_F16>(a, p, st) : prep<DT_BF16>(a, p, st);
}

hipError_t QP_CAT(launch_loss_tile_b, QP_BITS)(int dt, LossTileArgs a, hipStream_t st)
{
    return dt == DT_F32 ? tile<DT_F32>(a, st) : dt == DT_F16 ? tile<DT_F16>(a, st) : tile<DT_BF16>(a, st);
}

} // namespace qp
