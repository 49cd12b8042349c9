// ffn_act.h -- the gated activations of the dense feed-forward block (moe_act of include/moe.h).
#pragma once

#include "common.h"

namespace moe {

namespace {

// Reciprocal to 1 ulp (v_rcp_f32): the correctly rounded division takes ten instructions, and an
// epilogue's exponentials and divisions stand between two tiles of matrix work.
__device__ __forceinline__ float rcp(float z) { return __builtin_amdgcn_rcpf(z); }

__device__ __forceinline__ float sigm(float z) { return rcp(1.f + __expf(-z)); }

// tanh z = sign(z) (1 - e) / (1 + e), e = exp(-2 |z|); below 1/8, where 1 - e cancels, the odd series
// to z^7 (its next term is below 2^-29 of z there).
__device__ __forceinline__ float tanh_(float z)
{
    const float e = __expf(-2.f * fabsf(z)), z2 = z * z;
    const float s = z * (1.f + z2 * (-1.f / 3.f + z2 * (2.f / 15.f + z2 * (-17.f / 315.f))));
    return z2 < 1.f / 64.f ? s : copysignf((1.f - e) * rcp(1.f + e), z);
}

// The layer's activations (moe_act): h and its two derivatives.
template <int ACT>
__device__ __forceinline__ float gated(float g, float u)
{
    if constexpr (ACT == ACT_SITU) return 4.f * tanh_(0.25f * g) * sigm(g) * (25.f * tanh_(u * (1.f / 25.f)));
    return g * sigm(g) * u;
}

__device__ __forceinline__ float sech2(float z)
{
    const float e = __expf(-2.f * fabsf(z)), r = rcp(1.f + e);
    return 4.f * e * r * r;
}

template <int ACT>
__device__ __forceinline__ void gated_grad(float g, float u, float &h, float &dhdg, float &dhdu)
{
    const float s = sigm(g);
    if constexpr (ACT == ACT_SITU) {
        const float zg = 0.25f * g, zu = u * (1.f / 25.f);
        const float A = 4.f * tanh_(zg) * s, B = 25.f * tanh_(zu);
        h = A * B;
        dhdg = (sech2(zg) * s + A * (1.f - s)) * B;
        dhdu = A * sech2(zu);
        return;
    }
    const float silu = g * s;
    h = silu * u;
    dhdg = u * (s + silu * (1.f - s));
    dhdu = silu;
}

}  // namespace

}  // namespace moe
