// wgrad.hpp — the gradient of a quantized weight's scales and biases. With
// dW = dy^T x, dW[n, k] = sum_m dy[m, n] x[m, k], and w = q s' + b' of a group,
//   dscales[n, G] = sum_{k in G} q[n, k] dW[n, k],
//   dbiases[n, G] = sum_{k in G} dW[n, k].
// dW never leaves the registers: a wave's fp32 accumulators hold 128 whole k
// of each weight row, so every group (32, 64 or 128 k) closes inside a lane
// pair, the codes are multiplied in there, and only the two sums are stored.
// The matrix instruction's operand A is x (its rows are k) and B is dy (its
// columns are n): a lane then owns one weight row, and the k of its
// accumulators are known at compile time.
#pragma once

#include "common.hpp"
#include "model_ops.hpp"
#include "xgrad.hpp"

namespace qp {

// Sums the splits' partial sums [split][scales, biases][N * G] in split order.
template <int DT, bool SCALED>
__global__ __launch_bounds__(256) void wgrad_finish_kernel(const float* __restrict__ partial, int splits,
                                                           int64_t per_split, int64_t count, void* dscales,
                                                           void* dbiases, const float* scale)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < 2 * count; i += (int64_t)gridDim.x * 256) {
        const float sum = sum_splits(partial, splits, per_split, i), v = SCALED ? sum * *scale : sum;
        if (i < count)
            store_elem<DT>(dscales, i, v);
        else
            store_elem<DT>(dbiases, i - count, v);
    }
}

// One group's two sums of weight row n: to the outputs, or to the split's
// partial sums.
template <int DT, bool SCALED>
__device__ __forceinline__ void wgrad_store(const WgradArgs& a, const GradPlan& plan, int mat, int split,
                                            int64_t n, int64_t g, bool bias, float v)
{
    const int64_t groups = a.K / a.gs, count = a.N * groups, i = n * groups + g;
    if (plan.splits > 1)
        a.partial[(((int64_t)split * a.nmat + mat) * 2 + (bias ? 1 : 0)) * count + i] = v;
    else
        store_elem<DT>(bias ? a.dbiases[mat] : a.dscales[mat], i, SCALED ? v * *a.scale : v);
}

// Any type, size and alignment: fp32 products on the 32x32x2 matrix
// instruction. A block of four waves takes 128 k x 128 n, 16 m a step, each
// wave all 128 k of 32 weight rows. Bound by the instruction's 64 cycles where
// there are blocks enough; 130 rows of a 2048 x 768 weight 14 us, of which 4 are
// its products.
constexpr int WG_BK = 128, WG_BN = 128, WG_M = 16;

template <int BITS, int DT, bool SCALED>
__global__ __launch_bounds__(256) void wgrad_f32_kernel(WgradArgs a, GradPlan plan)
{
    __shared__ float xs[WG_M][WG_BK];
    __shared__ float ys[WG_M][WG_BN];
    const int tid = (int)threadIdx.x, lane = tid & 63, half = lane >> 5, c32 = lane & 31, wave = tid >> 6;
    const uint32_t tiles_k = (uint32_t)((a.K + WG_BK - 1) / WG_BK);
    const int64_t n0 = (int64_t)(blockIdx.x / tiles_k) * WG_BN, k0 = (int64_t)(blockIdx.x % tiles_k) * WG_BK;
    const int mat = (int)blockIdx.z, split = (int)blockIdx.y;
    const int64_t steps = (a.M + WG_M - 1) / WG_M;
    const int64_t lo = (int64_t)split * plan.per_split;
    int64_t hi = lo + plan.per_split;
    hi = hi < steps ? hi : steps;

    f32x16_t acc[4] = {};
    // No branch around a load (an index past the end is held inside and its
    // value dropped when it goes to LDS).
    using St = typename Elem<DT>::storage;
    St rx[8], ry[8];
    const int c = tid & 127;
    const bool k_in = k0 + c < a.K, n_in = n0 + c < a.N;
    const St* const px = static_cast<const St*>(a.x) + (k_in ? k0 + c : a.K - 1);
    const St* const py = static_cast<const St*>(a.dy[mat]) + (n_in ? n0 + c : a.N - 1);
    auto fetch = [&](int64_t step) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            int64_t m = step * WG_M + (tid >> 7) + 2 * i;
            m = m < a.M ? m : a.M - 1;
            rx[i] = px[m * a.K];
            ry[i] = py[m * a.dy_stride];
        }
    };
    if (lo < hi)
        fetch(lo);
    for (int64_t step = lo; step < hi; ++step) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool m_in = step * WG_M + (tid >> 7) + 2 * i < a.M;
            xs[(tid >> 7) + 2 * i][c] = live_or_zero(m_in && k_in, Elem<DT>::to_f32(rx[i]));
            ys[(tid >> 7) + 2 * i][c] = live_or_zero(m_in && n_in, Elem<DT>::to_f32(ry[i]));
        }
        __syncthreads();
        if (step + 1 < hi)
            fetch(step + 1);
#pragma unroll
        for (int kk = 0; kk < WG_M / 2; ++kk) {
            const float fy = ys[2 * kk + half][32 * wave + c32];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i] = __builtin_amdgcn_mfma_f32_32x32x2f32(xs[2 * kk + half][32 * i + c32], fy, acc[i], 0, 0, 0);
        }
    }
    // Accumulator r of tile i: k = k0 + 32 i + 8 (r / 4) + 4 half + r % 4 of
    // weight row n, so tile i is unit i of the row's codes here.
    const int64_t n = n0 + 32 * wave + c32;
    const int64_t row_words = a.K * BITS / 32;
    float ps[4], pb[4];
    // All the codes before any is used; units past the row's end are dropped below.
    uint32_t w[4][BITS];
    const uint32_t* const row = a.wq[mat] + (n < a.N ? n : a.N - 1) * row_words;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < BITS; ++j)
            w[i][j] = row[(k0 + 32 * i < a.K ? k0 / 32 + i : 0) * BITS + j];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float s = 0.0f, b = 0.0f;
        static_for<16>([&](auto R) {
            constexpr int r = decltype(R)::value, c = 8 * (r >> 2) + (r & 3);
            const uint32_t q = half ? unit_code<BITS, c + 4>(w[i]) : unit_code<BITS, c>(w[i]);
            s = __builtin_fmaf((float)q, acc[i][r], s);
            b += acc[i][r];
        });
        ps[i] = s + __shfl_xor(s, 32, 64);
        pb[i] = b + __shfl_xor(b, 32, 64);
    }
    if (n >= a.N)
        return;
    const int tiles = a.gs / 32;   // of a group: 1, 2 or 4
    for (int i = 0; i < 4 && k0 + 32 * i < a.K; i += tiles) {
        float v = 0.0f;
        static_for<4>([&](auto J) {
            constexpr int j = decltype(J)::value;
            if (j >= i && j < i + tiles)
                v += half ? pb[j] : ps[j];
        });
        wgrad_store<DT, SCALED>(a, plan, mat, split, n, (k0 + 32 * i) / a.gs, half != 0, v);
    }
}

} // namespace qp
