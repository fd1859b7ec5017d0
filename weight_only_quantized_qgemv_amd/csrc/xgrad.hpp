// xgrad.hpp — the input gradient of a quantized linear layer y = x W^T:
//   dx[m, k] = sum_n dy[m, n] w[n, k],   w = q s' + b',
// summed over one or two (dy, W) pairs (the gate and up projections of a
// gated block share their input), and the close that the gated block's down
// projection needs, where the product is dh and
//   h = act(g) u,  dg = dh u act'(g),  du = dh act(g)
// are written in its place.
#pragma once

#include "act.hpp"
#include "codes8.hpp"
#include "common.hpp"
#include "model_ops.hpp"

namespace qp {

inline size_t elem_size(int dt) { return dt == DT_F32 ? 4 : 2; }

template <int DT>
__device__ __forceinline__ float load_elem(const void* p, int64_t i)
{
    return Elem<DT>::to_f32(static_cast<const typename Elem<DT>::storage*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void store_elem(void* p, int64_t i, float v)
{
    static_cast<typename Elem<DT>::storage*>(p)[i] = Elem<DT>::from_f32(v);
}

// v times a factor that is on the device, where there is one.
__device__ __forceinline__ float scaled(float v, const float* scale)
{
    return scale != nullptr ? v * *scale : v;
}

// The result v of element i = m K + k of a call with sums: added to them, or stored.
template <int DT>
__device__ __forceinline__ void xgrad_add(const XgradArgs& a, int64_t i, float v)
{
    if (!a.first)
        v += a.sums[i];
    if (a.last)
        store_elem<DT>(a.out, i, scaled(v, a.scale));
    else
        a.sums[i] = v;
}

// The result v of element i = m K + k: stored, or closed as above (PIECES: added).
template <int DT, bool PIECES>
__device__ __forceinline__ void xgrad_store(const XgradArgs& a, int64_t i, float v)
{
    if constexpr (PIECES) {
        xgrad_add<DT>(a, i, v);
        return;
    }
    if (a.g == nullptr) {
        store_elem<DT>(a.out, i, v);
        return;
    }
    const float u = load_elem<DT>(a.u, i);
    float act, dact;
    act_grad_f32(a.act, load_elem<DT>(a.g, i), act, dact);
    store_elem<DT>(a.dg, i, v * u * dact);
    store_elem<DT>(a.du, i, v * act);
    if (a.h != nullptr)
        store_elem<DT>(a.h, i, act * u);
}

// The sum of element i's partial sums in split order, eight loads in flight.
__device__ __forceinline__ float sum_splits(const float* partial, int splits, int64_t stride, int64_t i)
{
    float v = 0.0f;
    for (int s = 0; s < splits; s += 8) {
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            p[j] = s + j < splits ? partial[(int64_t)(s + j) * stride + i] : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v += p[j];
    }
    return v;
}

// Sums the splits' partial sums and closes.
template <int DT, bool PIECES>
__global__ __launch_bounds__(256) void xgrad_finish_kernel(XgradArgs a, int splits)
{
    const int64_t total = a.M * a.K;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256)
        xgrad_store<DT, PIECES>(a, i, sum_splits(a.partial, splits, total, i));
}

// v, or zero: by its bits, since a select around a loaded value becomes a branch
// and a wait for each.
__device__ __forceinline__ float live_or_zero(bool live, float v)
{
    return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & (live ? ~0u : 0u));
}

// Any type, size and alignment: fp32 products on the 32x32x2 matrix
// instruction. A block of four waves computes 128 x 128 outputs, 32 n a step:
// dy goes to LDS as fp32 transposed, the weights dequantized, each thread two
// octets of codes. Bound by the instruction's 64 cycles (4096 a step): 2048 rows
// of a 14336 x 4096 weight 2150 us (112 TFLOP/s).
constexpr int XG_BM = 128, XG_BK = 128, XG_N = 32;

template <int BITS, int DT, bool PIECES>
__global__ __launch_bounds__(256) void xgrad_f32_kernel(XgradArgs a, GradPlan plan)
{
    using C8 = Codes8<BITS>;
    __shared__ float as[XG_N][XG_BM + 1];
    __shared__ __attribute__((aligned(16))) float bs[XG_N][XG_BK];
    const int tid = (int)threadIdx.x, lane = tid & 63, half = lane >> 5, c32 = lane & 31;
    const int wm = (tid >> 6) >> 1, wk = (tid >> 6) & 1;
    const uint32_t tiles_k = (uint32_t)((a.K + XG_BK - 1) / XG_BK);
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_k) * XG_BM, k0 = (int64_t)(blockIdx.x % tiles_k) * XG_BK;
    const int gs_log = 31 - __clz(a.gs);   // 32, 64 or 128
    const int64_t row_words = a.K * BITS / 32, groups = a.K >> gs_log;
    const int64_t steps = (a.N + XG_N - 1) / XG_N;       // of one pair
    const int64_t lo = (int64_t)blockIdx.y * plan.per_split;
    int64_t hi = lo + plan.per_split;
    hi = hi < steps * a.nmat ? hi : steps * a.nmat;

    f32x16_t acc[2][2] = {};
    // What a step needs, as loaded: no branch around a load (an index past the
    // end is held inside and its value dropped when it goes to LDS) and nothing
    // computed from one before the products that cover its latency.
    using St = typename Elem<DT>::storage;
    constexpr int NW = C8::NW;
    St ra[16], rs[2], rbias[2];
    uint32_t rw[2][NW];
    auto fetch = [&](int64_t step) {
        const int p = step >= steps;
        const int64_t n0 = (step - (p ? steps : 0)) * XG_N;
        const int64_t n = n0 + (tid & 31) < a.N ? n0 + (tid & 31) : a.N - 1;
        const St* const dy = static_cast<const St*>(a.dy[p]);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int64_t m = m0 + (tid >> 5) + 8 * i;
            ra[i] = dy[(m < a.M ? m : a.M - 1) * a.dy_stride + n];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int e = tid + 256 * j;
            const int64_t r = n0 + (e >> 4) < a.N ? n0 + (e >> 4) : a.N - 1;
            const int64_t k = k0 + 8 * (e & 15) < a.K ? k0 + 8 * (e & 15) : a.K - 8;
            const int oct = (int)(k >> 3);
            const uint32_t* const w = a.w[p].wq + r * row_words + C8::word(oct);
            rw[j][0] = w[0];
            if constexpr (NW == 2)
                rw[j][1] = w[C8::need2(oct) ? 1 : 0];
            const int64_t gi = r * groups + ((int)k >> gs_log);
            rs[j] = static_cast<const St*>(a.w[p].scales)[gi];
            rbias[j] = static_cast<const St*>(a.w[p].biases)[gi];
        }
    };
    auto stage = [&](int64_t step) {
        const int64_t n0 = (step - (step >= steps ? steps : 0)) * XG_N;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            as[tid & 31][(tid >> 5) + 8 * i] =
                live_or_zero(n0 + (tid & 31) < a.N && m0 + (tid >> 5) + 8 * i < a.M, Elem<DT>::to_f32(ra[i]));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int e = tid + 256 * j;
            const int64_t k = k0 + 8 * (e & 15);
            const bool live = n0 + (e >> 4) < a.N && k < a.K;
            float q[8];
            C8::to_f32(rw[j], (int)((live ? k : a.K - 8) >> 3), q);
            const float s = Elem<DT>::to_f32(rs[j]), b = Elem<DT>::to_f32(rbias[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                q[i] = live ? __builtin_fmaf(q[i], s, b) : 0.0f;
            f32x4_t* d = reinterpret_cast<f32x4_t*>(&bs[e >> 4][8 * (e & 15)]);
            d[0] = f32x4_t{q[0], q[1], q[2], q[3]};
            d[1] = f32x4_t{q[4], q[5], q[6], q[7]};
        }
    };
    if (lo < hi)
        fetch(lo);
    for (int64_t step = lo; step < hi; ++step) {
        __syncthreads();
        stage(step);
        __syncthreads();
        if (step + 1 < hi)
            fetch(step + 1);
#pragma unroll
        for (int kk = 0; kk < XG_N / 2; ++kk) {
            float fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fa[i] = as[2 * kk + half][wm * 64 + 32 * i + c32];
                fb[i] = bs[2 * kk + half][wk * 64 + 32 * i + c32];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[i], fb[j], acc[i][j], 0, 0, 0);
        }
    }
    // One loop for each close: chosen inside it, the close's code would lie
    // between two stores of the partial sums, which then wait for instructions.
    auto each = [&](auto&& f) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int64_t m = m0 + wm * 64 + 32 * i + 8 * (r >> 2) + 4 * half + (r & 3);
                    const int64_t k = k0 + wk * 64 + 32 * j + c32;
                    if (m < a.M && k < a.K)
                        f(m * a.K + k, acc[i][j][r]);
                }
    };
    if (plan.splits > 1) {
        float* const part = a.partial + (int64_t)blockIdx.y * a.M * a.K;
        each([&](int64_t i, float v) { part[i] = v; });
    } else if constexpr (PIECES) {
        each([&](int64_t i, float v) { xgrad_add<DT>(a, i, v); });
    } else if (a.g == nullptr) {
        each([&](int64_t i, float v) { store_elem<DT>(a.out, i, v); });
    } else {
        each([&](int64_t i, float v) { xgrad_store<DT, false>(a, i, v); });
    }
}

} // namespace qp
