// act.hpp — the activations of the gated feed-forward block and their
// derivatives, in fp32.
//   SiLU:       a(z) = z s,  s = 1 / (1 + e^-z)
//   GELU, tanh: a(z) = z (1 + tanh y) / 2 = z s(2y),  y = sqrt(2/pi) (z + 0.044715 z^3)
// Both are z s(p) with p = z or 2y, so  a'(z) = s + z s (1 - s) p'.
// (1 - s) is formed as s(-p), not by subtraction, and a product s (1 - s) that
// has vanished makes its term zero whatever z is (z may have overflowed).
#pragma once

#include "common.hpp"
#include "model_ops.hpp"

namespace qp {

template <int ACT> __device__ __forceinline__ float act_arg(float z)
{
    if constexpr (ACT == ACT_SILU)
        return z;
    else
        return 1.5957691216057308f * (z + 0.044715f * z * z * z);
}

template <int ACT> __device__ __forceinline__ float act_f32(float z)
{
    return z / (1.0f + expf(-act_arg<ACT>(z)));
}

// a(z) and a'(z).
template <int ACT> __device__ __forceinline__ void act_grad_f32(float z, float& a, float& da)
{
    const float p = act_arg<ACT>(z);
    const float s = 1.0f / (1.0f + expf(-p)), t = 1.0f / (1.0f + expf(p));
    const float dp = ACT == ACT_SILU ? 1.0f : 1.5957691216057308f * (1.0f + 0.134145f * z * z);
    const float st = s * t;
    a = z * s;
    da = s + (st == 0.0f ? 0.0f : z * st * dp);
}

__device__ __forceinline__ float act_f32(int act, float z)
{
    return act == ACT_SILU ? act_f32<ACT_SILU>(z) : act_f32<ACT_GELU_TANH>(z);
}
__device__ __forceinline__ void act_grad_f32(int act, float z, float& a, float& da)
{
    if (act == ACT_SILU)
        act_grad_f32<ACT_SILU>(z, a, da);
    else
        act_grad_f32<ACT_GELU_TANH>(z, a, da);
}

} // namespace qp
