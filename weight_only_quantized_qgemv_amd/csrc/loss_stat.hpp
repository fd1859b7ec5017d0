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

} // namespace qp
