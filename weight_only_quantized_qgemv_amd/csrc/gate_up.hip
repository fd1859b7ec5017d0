// gate_up.hip — the fused first half of the gated feed-forward block,
//   h = act(x Wg^T) * (x Wu^T),
// both projections, the activation and the product in one launch, for 16-bit
// activations: the row kernel at one and two rows (rowstream.hpp), the skinny
// matrix-core kernel up to 16 (skinny.hpp), the tile kernel beyond
// (gemm_core.hpp). Each closes h from its fp32 sums, and stores the two products
// beside it where a backward pass follows: h is the same with and without them.
// Compiled once per bit width (QP_BITS).
#include <algorithm>

#include "gemm_core.hpp"
#include "model_ops.hpp"
#include "rowstream.hpp"
#include "skinny.hpp"

namespace qp {

namespace {

constexpr int64_t k2GB = int64_t(1) << 31;

template <int BITS, int DT, int MT, int UPL, int KL>
hipError_t run_rows(const GateUpArgs& a, hipStream_t st)
{
    constexpr int WPB = 4, D = rowstream_depth<BITS, UPL * 2, MT>(), ROWS = WPB * (64 / KL) * D;
    RowStreamArgs k{};
    k.x = a.x;
    k.wq = a.gate.wq; k.scales = a.gate.scales; k.biases = a.gate.biases;
    k.up_wq = a.up.wq; k.up_scales = a.up.scales; k.up_biases = a.up.biases;
    k.y = a.h;
    k.M = (int)a.M; k.N = (int)a.N; k.K = (int)a.K; k.gs = a.gs;
    k.units_row = (uint32_t)(a.K / 32);
    k.act = a.act;
    k.saved[0] = a.saved[0]; k.saved[1] = a.saved[1];
    const int64_t blocks = std::min<int64_t>((a.N + ROWS - 1) / ROWS, 4096);
    if ((a.K / a.gs) % 2 == 0 && reinterpret_cast<uintptr_t>(a.gate.scales) % 4 == 0 &&
        reinterpret_cast<uintptr_t>(a.gate.biases) % 4 == 0 && reinterpret_cast<uintptr_t>(a.up.scales) % 4 == 0 &&
        reinterpret_cast<uintptr_t>(a.up.biases) % 4 == 0)
        hipLaunchKernelGGL((qgemv_rowstream_kernel<BITS, DT, MT, UPL, WPB, true, KL, 2>), dim3((unsigned)blocks),
                           dim3(64 * WPB), 0, st, k);
    else
        hipLaunchKernelGGL((qgemv_rowstream_kernel<BITS, DT, MT, UPL, WPB, false, KL, 2>), dim3((unsigned)blocks),
                           dim3(64 * WPB), 0, st, k);
    return hipGetLastError();
}

// Units per lane as the row needs them, up to four (two activation rows: two):
// both matrices' codes and the activation slices share the registers.
template <int BITS, int DT, int MT>
hipError_t run_rows_upl(const GateUpArgs& a, hipStream_t st, bool* done)
{
    const int64_t units = a.K / 32;
    *done = true;
    if (units <= 32) return run_rows<BITS, DT, MT, 1, 32>(a, st);
    if (units <= 64) return run_rows<BITS, DT, MT, 1, 64>(a, st);
    if (units <= 128) return run_rows<BITS, DT, MT, 2, 64>(a, st);
    if constexpr (MT == 1) {
        if (units <= 192) return run_rows<BITS, DT, MT, 3, 64>(a, st);
        if (units <= 256) return run_rows<BITS, DT, MT, 4, 64>(a, st);
    }
    *done = false;
    return hipSuccess;
}

template <int BITS, int DT>
hipError_t run_skinny(const GateUpArgs& a, hipStream_t st)
{
    GemvKernelArgs k{};
    k.x = a.x;
    k.top_k = 1;
    k.outer = a.K;
    k.M = (int)a.M;
    k.wq[0] = a.gate.wq; k.scales[0] = a.gate.scales; k.biases[0] = a.gate.biases;
    k.wq[1] = a.up.wq; k.scales[1] = a.up.scales; k.biases[1] = a.up.biases;
    k.R = a.N; k.K = a.K; k.gs = a.gs;
    k.out = a.h;
    k.out_bytes = (uint32_t)(a.M * a.N * 2);
    k.x_bytes = (uint32_t)(a.M * a.K * 2);
    k.act = a.act;
    k.saved[0] = a.saved[0]; k.saved[1] = a.saved[1];
    SkinnyShape sh{};
    dim3 grid;
    skinny_dense_shape(a.N, a.K, &sh, &grid);
    return skinny_launch<BITS, DT, 2>(k, sh, grid, st);
}

template <int BITS, int DT, int BM, int BN, int NT, int WMW>
hipError_t run_tiles(const GateUpArgs& a, hipStream_t st)
{
    constexpr int NA = 3, NC = 4;
    constexpr int LDS = gemm::lds_bytes<BITS, BM, BN, NT, NA, NC>();
    static_assert(LDS <= 160 * 1024, "LDS budget");
    const void* kern = reinterpret_cast<const void*>(
        &gemm::qgemm_tile_kernel<BITS, DT, BM, BN, NT, WMW, 2, false, NA, NC>);
    static std::atomic<uint64_t> lds{0};   // per instantiation
    if (hipError_t e = allow_lds(lds, kern, LDS); e != hipSuccess)
        return e;
    GemmArgs g{};
    g.x = a.x;
    g.wq[0] = a.gate.wq; g.scales[0] = a.gate.scales; g.biases[0] = a.gate.biases;
    g.wq[1] = a.up.wq; g.scales[1] = a.up.scales; g.biases[1] = a.up.biases;
    g.y = a.h;
    g.M = (int)a.M; g.N = (int)a.N; g.K = (int)a.K; g.gs = a.gs;
    g.x_bytes = (uint32_t)(a.M * a.K * 2);
    g.y_bytes = (uint32_t)(a.M * a.N * 2);
    g.sb_bytes = (uint32_t)((a.N * (a.K / a.gs) * 2 + 3) & ~int64_t(3));
    g.tiles_n = (int)((a.N + BN / 2 - 1) / (BN / 2));
    g.tiles = (int)((a.M + BM - 1) / BM) * g.tiles_n;
    g.per_xcd = (g.tiles + 7) / 8;
    g.act = a.act;
    g.saved[0] = a.saved[0]; g.saved[1] = a.saved[1];
    hipLaunchKernelGGL((gemm::qgemm_tile_kernel<BITS, DT, BM, BN, NT, WMW, 2, false, NA, NC>), dim3(g.per_xcd * 8),
                       dim3(NT), LDS, st, g);
    return hipGetLastError();
}

template <int BITS, int DT>
hipError_t run(const GateUpArgs& a, hipStream_t st, bool* done)
{
    *done = false;
    if (!aligned16(a.x) || a.N * (a.K * BITS / 8) >= k2GB || a.N * (a.K / a.gs) * 2 >= k2GB - 4 ||
        a.M * a.N * 2 >= k2GB || a.M * a.K * 2 >= k2GB || a.K >= (1 << 30))
        return hipSuccess;
    if (a.M <= 16) {
        // The row kernel where its registers hold the rows' slices. One row beyond
        // (the whole block, 4-bit, d_ff 8192): 9216 39.9 us on the skinny kernel,
        // two products and a third launch 40.1; 16384 61.9 and 64.2; 17408 65 and 702.
        if (a.M <= 2) {
            hipError_t e = a.M == 1 ? run_rows_upl<BITS, DT, 1>(a, st, done) : run_rows_upl<BITS, DT, 2>(a, st, done);
            if (e != hipSuccess || *done)
                return e;
        }
        *done = true;
        return run_skinny<BITS, DT>(a, st);
    }
    const bool dwords = (reinterpret_cast<uintptr_t>(a.gate.scales) | reinterpret_cast<uintptr_t>(a.gate.biases) |
                         reinterpret_cast<uintptr_t>(a.up.scales) | reinterpret_cast<uintptr_t>(a.up.biases)) % 4 == 0;
    if (a.K % gemm::BK != 0 || !dwords)
        return hipSuccess;
    *done = true;
    // Measured with 4-bit codes, the whole block's time. Up to 128 rows tiles of
    // 64: 128 rows of a 2048 x 5632 block 113 us, with tiles of 256 x 128 124.
    // 256 x 256 tiles where there are more than 128, so that half as wide ones
    // would not fit the 256 CUs at once: 512 rows of 4096 x 14336 (224 tiles)
    // 326 us, half as wide 355; 256 rows (112 tiles) 300 against 278. Their
    // stages fit the LDS up to 4-bit codes.
    if (a.M <= 128)
        return run_tiles<BITS, DT, 64, 256, 256, 1>(a, st);
    if constexpr (BITS <= 4) {
        if (((a.M + 255) / 256) * ((a.N + 127) / 128) > 128)
            return run_tiles<BITS, DT, 256, 256, 512, 2>(a, st);
    }
    return run_tiles<BITS, DT, 256, 128, 256, 2>(a, st);
}

template <int BITS, int DT, int BM, int BN, int WMW, int NMAT>
hipError_t run_split(const FfnSplitArgs& a, hipStream_t st)
{
    constexpr int NA = 3, NC = 4, NT = 256;
    constexpr int LDS = gemm::lds_bytes<BITS, BM, BN, NT, NA, NC>();
    static_assert(LDS <= 160 * 1024, "LDS budget");
    const void* kern = reinterpret_cast<const void*>(
        &gemm::qgemm_tile_kernel<BITS, DT, BM, BN, NT, WMW, NMAT, false, NA, NC, 0, true>);
    static std::atomic<uint64_t> lds{0};   // per instantiation
    if (hipError_t e = allow_lds(lds, kern, LDS); e != hipSuccess)
        return e;
    GemmArgs g{};
    g.x = a.x;
    for (int t = 0; t < 2; ++t) {
        const QWeight& w = a.w[t < NMAT ? t : 0];
        g.wq[t] = w.wq; g.scales[t] = w.scales; g.biases[t] = w.biases;
    }
    g.M = (int)a.M; g.N = (int)a.N; g.K = (int)a.K; g.gs = a.gs;
    g.x_bytes = (uint32_t)(a.M * a.K * 2);
    g.sb_bytes = (uint32_t)((a.N * (a.K / a.gs) * 2 + 3) & ~int64_t(3));
    g.tiles_n = (int)((a.N + BN / NMAT - 1) / (BN / NMAT));
    g.tiles = (int)((a.M + BM - 1) / BM) * g.tiles_n;
    g.per_xcd = (g.tiles + 7) / 8;
    g.partial = a.partial;
    g.per_split = a.plan.per_split;
    g.wk = (int)a.wk;
    hipLaunchKernelGGL((gemm::qgemm_tile_kernel<BITS, DT, BM, BN, NT, WMW, NMAT, false, NA, NC, 0, true>),
                       dim3(g.per_xcd * 8, (unsigned)a.plan.splits), dim3(NT), LDS, st, g);
    return hipGetLastError();
}

template <int DT> hipError_t run_split_dt(const FfnSplitArgs& a, hipStream_t st)
{
    if (a.plan.tile == 64)
        return a.nmat == 2 ? run_split<QP_BITS, DT, 64, 256, 1, 2>(a, st) : run_split<QP_BITS, DT, 64, 256, 1, 1>(a, st);
    return a.nmat == 2 ? run_split<QP_BITS, DT, 256, 128, 2, 2>(a, st) : run_split<QP_BITS, DT, 256, 128, 2, 1>(a, st);
}

} // namespace

hipError_t QP_CAT(launch_ffn_split_b, QP_BITS)(const FfnSplitArgs& a, hipStream_t st)
{
    switch (a.dt) {
    case DT_F16: return run_split_dt<DT_F16>(a, st);
    case DT_BF16: return run_split_dt<DT_BF16>(a, st);
    }
    return hipErrorInvalidValue;
}

hipError_t QP_CAT(launch_gate_up_b, QP_BITS)(const GateUpArgs& a, hipStream_t st, bool* done)
{
    switch (a.dt) {
    case DT_F16: return run<QP_BITS, DT_F16>(a, st, done);
    case DT_BF16: return run<QP_BITS, DT_BF16>(a, st, done);
    }
    *done = false;
    return hipSuccess;
}

} // namespace qp
