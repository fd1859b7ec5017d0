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
    static std::atomic<uint64_t> lds{0};   // per instantiation
    if (hipError_t e = allow_lds(lds, kern, LDS); e != hipSuccess)
        return e;
    const int64_t tiles_k = (a.K + BN - 1) / BN, tiles = (a.M + BM - 1) / BM * tiles_k;
    const int per_xcd = (int)((tiles + 7) / 8);
    if (!grid_fits((int64_t)per_xcd * 8, 2 * BN))
        return hipErrorInvalidConfiguration;
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
        if (!grid_fits(tiles, 256))
            return hipErrorInvalidConfiguration;
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
// The plan takes the least of an estimate, in us, over the tiles and the pieces
// of the contraction: rounds of resident blocks times a piece's steps, the
// partial sums' way out and back (8 TB/s: mostly caches), a launch for their
// sum, and what a block costs besides its steps. Measured against it, 4-bit,
// bf16, contraction 14336 to 4096 columns: 64 rows tile 64 27 us, 128 32, 256
// 41; 128 rows 40, 36.6, 44; 1024 rows 218, 167, 131; contraction 4096, 512
// rows: 49, 37.8, 43.7.
GradPlan xgrad_plan(int64_t m, int64_t n, int64_t k, int nmat, bool tile_kernels)
{
    struct Tile {
        int tile;
        int64_t bm, bn, step, resident;
        double us, fixed;
    };
    constexpr Tile kTiles[] = {{1, 256, 256, gradtile::STEP, 256, 1.25, 12.0}, {2, 128, 128, gradtile::STEP, 512, 1.3, 3.0},
                               {3, 64, 128, gradtile::STEP, 512, 0.95, 2.0}, {0, XG_BM, XG_BK, XG_N, 512, 4.0, 3.0}};
    GradPlan p{};
    double best = -1.0;
    for (const Tile& t : kTiles) {
        if ((t.tile != 0) != tile_kernels)
            continue;
        const int64_t tiles = std::max<int64_t>(((m + t.bm - 1) / t.bm) * ((k + t.bn - 1) / t.bn), 1);
        const int64_t steps = nmat * ((n + t.step - 1) / t.step);
        for (int64_t want = 1; want <= 64 && (want == 1 || 4 * want <= steps); ++want) {
            const int64_t per = std::max<int64_t>((steps + want - 1) / want, 1);
            const int64_t splits = std::max<int64_t>((steps + per - 1) / per, 1);
            double us = (double)((tiles * splits + t.resident - 1) / t.resident) * (double)per * t.us + t.fixed;
            if (splits > 1)
                us += 4.0 + (double)splits * (double)m * (double)k * 8.0 / 8e6;
            if (best < 0.0 || us < best) {
                best = us;
                p.tile = t.tile;
                p.per_split = per;
                p.splits = (int)splits;
            }
        }
    }
    p.partial_bytes = p.splits > 1 ? (size_t)p.splits * (size_t)m * (size_t)k * 4 : 0;
    return p;
}
#endif

} // namespace qp
