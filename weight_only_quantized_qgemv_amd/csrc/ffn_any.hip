// ffn_any.hip — the gated block's products for what the other kernels do not
// take: fp32 activations of more than one row, and 16-bit ones of more than 16
// rows that contract over 32 or whose weights take 2 GB or more. y = x W^T on the
// fp32 32x32x2 matrix instruction, any size and alignment, nothing rounded
// before y (or before the fp32 sums that another launch closes).
// Compiled once per bit width (QP_BITS).
#include <algorithm>

#include "codes8.hpp"
#include "common.hpp"
#include "model_ops.hpp"
#include "xgrad.hpp"

namespace qp {

namespace {

constexpr int AN_N = 128, AN_K = 32;   // weight rows a block, k a step

// Four waves, each 32 weight rows times 32 FM activation rows. A lane's half of
// the wave takes 16 consecutive k of the step (any pairing of k will do, as
// long as both operands have it), so it dequantizes just its own codes, into
// registers; the activations go through LDS, shared by the waves, in rows of
// 36 floats (16 lanes' 16-byte reads fall on all banks). Loads run D steps
// ahead: four in the kernel for up to 32 rows, where the weights' latency shows,
// one in that for 128, bound by the matrix instructions (16 FM of 64 cycles a
// step). A 4096 x 14336 block in fp32, 4-bit: 2 to 32 rows 149 to 157 us, 128
// rows 456, 2048 rows 5881 (123 TFLOP/s; a large fp32 library product reaches 154).
template <int BITS, int DT, int FM, int D>
__global__ __launch_bounds__(256) void ffn_any_kernel(FfnAnyArgs a)
{
    using C8 = Codes8<BITS>;
    using St = typename Elem<DT>::storage;
    constexpr int BM = 32 * FM, NW = C8::NW, NX = BM / 8, ROW = AN_K + 4;
    __shared__ __attribute__((aligned(16))) float xs[2][BM][ROW];
    const int tid = (int)threadIdx.x, lane = tid & 63, half = lane >> 5, c32 = lane & 31, wave = tid >> 6;
    const uint32_t tiles_m = (uint32_t)((a.M + BM - 1) / BM);
    const int64_t m0 = (int64_t)(blockIdx.x % tiles_m) * BM, n0 = (int64_t)(blockIdx.x / tiles_m) * AN_N;
    const int64_t n = n0 + 32 * wave + c32, row = n < a.N ? n : a.N - 1;
    const int gs_log = 31 - __clz(a.gs);   // 32, 64 or 128
    const int64_t groups = a.K >> gs_log;
    const int steps = (int)(a.K / AN_K), lo = (int)blockIdx.y * a.plan.per_split;
    const int hi = lo + a.plan.per_split < steps ? lo + a.plan.per_split : steps;

    const uint32_t* const wq = a.w.wq + row * (a.K * BITS / 32);
    const St* const ps = static_cast<const St*>(a.w.scales) + row * groups;
    const St* const pb = static_cast<const St*>(a.w.biases) + row * groups;
    const St* px[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        const int64_t m = m0 + (tid >> 5) + 8 * i;
        px[i] = static_cast<const St*>(a.x) + (m < a.M ? m : a.M - 1) * a.K + (tid & 31);
    }

    // A step as loaded; rows past the ends repeat the last one and are not stored.
    struct Raw {
        St x[NX], s, b;
        uint32_t w[2][NW];
    };
    Raw ring[D];
    auto fetch = [&](int step, Raw& r) {
        step = step < hi ? step : hi - 1;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const int oct = 4 * step + 2 * half + o;
            r.w[o][0] = wq[C8::word(oct)];
            if constexpr (NW == 2)
                r.w[o][1] = wq[C8::word(oct) + (C8::need2(oct) ? 1 : 0)];
        }
        const int g = (step * AN_K) >> gs_log;
        r.s = ps[g];
        r.b = pb[g];
#pragma unroll
        for (int i = 0; i < NX; ++i)
            r.x[i] = px[i][(int64_t)step * AN_K];
    };

    f32x16_t acc[FM] = {};
    static_for<D>([&](auto J) { fetch(lo + (int)J, ring[J]); });
    for (int base = lo; base < hi; base += D) {
        static_for<D>([&](auto J) {
            constexpr int j = decltype(J)::value;
            const int step = base + j;
            if (step >= hi)   // uniform
                return;
            Raw& r = ring[j];
            float(&xb)[BM][ROW] = xs[(step - lo) & 1];
#pragma unroll
            for (int i = 0; i < NX; ++i)
                xb[(tid >> 5) + 8 * i][tid & 31] = Elem<DT>::to_f32(r.x[i]);
            float w[2][8];
            const float s = Elem<DT>::to_f32(r.s), b = Elem<DT>::to_f32(r.b);
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                C8::to_f32(r.w[o], 4 * step + 2 * half + o, w[o]);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[o][i] = __builtin_fmaf(w[o][i], s, b);
            }
            __syncthreads();
            fetch(step + D, r);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f32x4_t xv[FM];
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    xv[i] = *reinterpret_cast<const f32x4_t*>(&xb[32 * i + c32][16 * half + 4 * q]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int i = 0; i < FM; ++i)
                        acc[i] = __builtin_amdgcn_mfma_f32_32x32x2f32(xv[i][e], w[q / 2][4 * (q % 2) + e], acc[i], 0, 0, 0);
            }
        });
    }
    // Accumulator r of tile i: row m0 + 32 i + 8 (r / 4) + 4 half + r % 4, weight row n.
    auto each = [&](auto&& f) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int64_t m = m0 + 32 * i + 8 * (r >> 2) + 4 * half + (r & 3);
                if (m < a.M && n < a.N)
                    f(m * a.N + n, acc[i][r]);
            }
    };
    if (a.partial != nullptr) {
        float* const part = a.partial + (int64_t)blockIdx.y * a.partial_stride;
        each([&](int64_t i, float v) { part[i] = v; });
    } else {
        each([&](int64_t i, float v) { store_elem<DT>(a.y, i, v); });
    }
}

template <int DT> hipError_t run(const FfnAnyArgs& a, hipStream_t st)
{
    const int64_t bm = a.plan.tile, tiles = ((a.M + bm - 1) / bm) * ((a.N + AN_N - 1) / AN_N);
    if (!grid_fits(tiles, 256))
        return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)tiles, (unsigned)a.plan.splits);
    if (bm == 32)
        hipLaunchKernelGGL((ffn_any_kernel<QP_BITS, DT, 1, 4>), grid, dim3(256), 0, st, a);
    else if (bm == 64)
        hipLaunchKernelGGL((ffn_any_kernel<QP_BITS, DT, 2, 2>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((ffn_any_kernel<QP_BITS, DT, 4, 1>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

} // namespace

hipError_t QP_CAT(launch_ffn_any_b, QP_BITS)(const FfnAnyArgs& a, hipStream_t st)
{
    switch (a.dt) {
    case DT_F32: return run<DT_F32>(a, st);
    case DT_F16: return run<DT_F16>(a, st);
    case DT_BF16: return run<DT_BF16>(a, st);
    }
    return hipErrorInvalidValue;
}

} // namespace qp
