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

} // namespace qp
