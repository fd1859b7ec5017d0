// loss_rows.hip — logits of up to 16 rows for the cross entropy, as fp32: the decode
// kernels of qmatmul (rowstream.hpp, skinny.hpp, skinny4.hpp), which stream the weights once
// and keep the codes exact, with their sums stored unrounded. Compiled once per bit width
// (QP_BITS).
#include <algorithm>

#include "model_ops.hpp"
#include "rowstream.hpp"
#include "skinny4.hpp"
#include "train_ops.hpp"

namespace qp {

namespace {

template <int DT, int MT, int UPL, int KL>
hipError_t run_rows(const GemvArgs& a, hipStream_t st)
{
    constexpr int WPB = 4, ROWS = WPB * (64 / KL) * rowstream_depth<QP_BITS, UPL, MT>();
    RowStreamArgs k{};
    k.x = a.x;
    k.wq = a.wq; k.scales = a.scales; k.biases = a.biases;
    k.y = a.y;
    k.M = (int)a.M; k.N = (int)a.N; k.K = (int)a.K; k.gs = a.gs;
    k.units_row = (uint32_t)(a.K / 32);
    const dim3 grid((unsigned)std::min<int64_t>((a.N + ROWS - 1) / ROWS, 4096));
    // Scales and biases as whole dword-aligned rows when a row has an even number of
    // groups (and their arrays are dword-aligned).
    const uintptr_t sb = reinterpret_cast<uintptr_t>(a.scales) | reinterpret_cast<uintptr_t>(a.biases);
    if ((a.K / a.gs) % 2 == 0 && sb % 4 == 0)
        hipLaunchKernelGGL((qgemv_rowstream_kernel<QP_BITS, DT, MT, UPL, WPB, true, KL, 1, DT_F32>), grid, dim3(64 * WPB),
                           0, st, k);
    else
        hipLaunchKernelGGL((qgemv_rowstream_kernel<QP_BITS, DT, MT, UPL, WPB, false, KL, 1, DT_F32>), grid, dim3(64 * WPB),
                           0, st, k);
    return hipGetLastError();
}

// One and two rows, as units per lane fit the registers; false in *done where they do not.
template <int DT, int MT>
hipError_t rows_upl(const GemvArgs& a, hipStream_t st, bool* done)
{
    const int64_t units = a.K / 32;
    *done = true;
    if (units <= 32) return run_rows<DT, MT, 1, 32>(a, st);
    if (units <= 64) return run_rows<DT, MT, 1, 64>(a, st);
    if (units <= 128) return run_rows<DT, MT, 2, 64>(a, st);
    if (units <= 256) return run_rows<DT, MT, 4, 64>(a, st);
    *done = false;
    return hipSuccess;
}

template <int DT> hipError_t run(const GemvArgs& a, hipStream_t st)
{
    if (a.M <= 2 && a.N * (a.K * QP_BITS / 8) < (int64_t(1) << 31)) {
        bool done = false;
        hipError_t e = a.M == 1 ? rows_upl<DT, 1>(a, st, &done) : rows_upl<DT, 2>(a, st, &done);
        if (e != hipSuccess || done)
            return e;
    }
    GemvKernelArgs k{};
    k.x = a.x;
    k.top_k = 1;
    k.outer = a.K;
    k.M = (int)a.M;
    k.wq[0] = k.wq[1] = a.wq;
    k.scales[0] = k.scales[1] = a.scales;
    k.biases[0] = k.biases[1] = a.biases;
    k.R = a.N; k.K = a.K; k.gs = a.gs;
    k.out = a.y;
    k.out_bytes = (uint32_t)(a.M * a.N * 4);
    k.x_bytes = (uint32_t)(a.M * a.K * 2);
    SkinnyShape sh{};
    dim3 grid;
    skinny_dense_shape(a.N, a.K, &sh, &grid);
    if constexpr (QP_BITS != 8) {
        if (skinny4_takes<QP_BITS>(a, sh))
            return skinny4_launch<QP_BITS, DT, DT_F32>(k, sh, grid, st);
    }
    return skinny_launch<QP_BITS, DT, 1, DT_F32>(k, sh, grid, st);
}

} // namespace

hipError_t QP_CAT(launch_loss_rows_b, QP_BITS)(const GemvArgs& a, hipStream_t st)
{
    return a.dt == DT_F16 ? run<DT_F16>(a, st) : run<DT_BF16>(a, st);
}

} // namespace qp
