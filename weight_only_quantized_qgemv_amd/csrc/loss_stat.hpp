// loss_stat.hpp — what a part of a row's logits is reduced to, for the cross entropy.
#pragma once

#include "common.hpp"

namespace qp {

struct Stat {
    float top, sum;   // the largest logit, the sum of exp(z - top)
};

// Two parts' statistics as one (an empty part: -infinity, 0).
__device__ __forceinline__ Stat join_stats(Stat a, Stat b)
{
    const float top = fmaxf(a.top, b.top);
    if (top == -__builtin_inff())
        return Stat{top, a.sum + b.sum};   // nothing, or NaN
    return Stat{top, a.sum * expf(a.top - top) + b.sum * expf(b.top - top)};
}

// The statistics of a wave's 64 lanes (or, LANES = 16, of 16 in a row), in all of them:
// the maximum, and then the sums once on its scale.
template <int LANES = 64> __device__ __forceinline__ Stat wave_stat(Stat s)
{
    auto over = [](float v, auto f) {
        v = f(v, dpp_f32<0xB1>(v));
        v = f(v, dpp_f32<0x4E>(v));
        v = f(v, dpp_f32<0x141>(v));
        v = f(v, dpp_f32<0x140>(v));
        if constexpr (LANES == 64) {
            const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
            v = f(__uint_as_float(x[0]), __uint_as_float(x[1]));
            const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
            v = f(__uint_as_float(y[0]), __uint_as_float(y[1]));
        }
        return v;
    };
    const float top = over(s.top, [](float a, float b) { return fmaxf(a, b); });
    const float own = top == -__builtin_inff() ? s.sum : s.sum * expf(s.top - top);   // (nothing, or NaN)
    return Stat{top, over(own, [](float a, float b) { return a + b; })};
}

// The factor that makes the rows' largest |dloss| 2^14, and what takes it out of the
// sums again (scale[0] and [1]), by one block of 256 threads. dz is the products' 16-bit
// operand: most of it is p - 1 or a small p times one and the same dloss, whose own
// rounding would not average out (2048 rows, a mean over 1843 of them, in bf16: the
// gradients 0.0040 of their size off 64 bits, with the factor 0.0024); and in fp16 a mean
// over many rows would leave the normal range (2^-14) for a token of probability 1e-2
// already. It is one factor for all rows, since dW sums over them: in fp16 a dz below 2^-28
// of the largest |dloss| is subnormal, so a row of a far smaller dloss than another's keeps
// fewer digits of its small probabilities.
__device__ __forceinline__ void dz_factor(const float* __restrict__ dloss, int64_t m, const int32_t* __restrict__ targets,
                                          int64_t vocab, float* __restrict__ scale)
{
    __shared__ float room[4];
    float top = 0.0f;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < m; i += 256) {
        const float g = fabsf(dloss[i]);
        const int32_t t = targets[i];
        top = fmaxf(top, t >= 0 && t < vocab && g < __builtin_inff() ? g : 0.0f);
    }
    top = wave_stat(Stat{top, 0.0f}).top;
    if ((threadIdx.x & 63) == 0)
        room[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x != 0)
        return;
    for (int w = 1; w < 4; ++w)
        top = fmaxf(top, room[w]);
    top = top > 0.0f ? fmaxf(top, 0x1p-100f) : 16384.0f;   // (both factors stay finite)
    scale[0] = 16384.0f / top;
    scale[1] = top / 16384.0f;
}

} // namespace qp
