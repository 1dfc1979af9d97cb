// The gated feed-forward block ("transition") of a pair, MSA or single
// representation: shared arithmetic.
//
//     G = X Wg^T,  U = X Wu^T,  H = act(G) * U,  Y = H Wd^T
//     dH = dY Wd,  dG = dH * U * act'(G),  dU = dH * act(G)
//     dX = dG Wg + dU Wu,  dWg = dG^T X,  dWu = dU^T X,  dWd = dY^T H
//
// with X, Y [M, C], Wg and Wu [F, C], Wd [C, F].  Every product is accumulated
// in fp32 and the activation is computed in fp32.  With 16-bit inputs H, dG and
// dU are rounded once to the input type, because they are operands of the next
// product's 16-bit MMA; dH never is.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "common.cuh"

namespace evo {

// 1 / (1 + e^-g).  __expf and __fdividef are within 2 ulp or so of fp32 here;
// e^-g overflows to inf below g = -88, which gives 0, the right limit.
__device__ __forceinline__ float tr_sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// act(g) and its derivative.  silu: g s, s (1 + g (1 - s)) with s = sigmoid(g);
// gelu: g Phi(g), Phi(g) + g phi(g), Phi and phi the normal distribution and density.
template <int ACT>
__device__ __forceinline__ float tr_act(float g) {
    if constexpr (ACT == EVO_ACT_SILU) {
        return g < -88.0f ? 0.0f : g * tr_sigmoid(g);
    } else {
        return 0.5f * g * erfcf(-0.70710678118654752f * g);
    }
}

template <int ACT>
__device__ __forceinline__ void tr_act_grad(float g, float& a, float& da) {
    if constexpr (ACT == EVO_ACT_SILU) {
        const float s = g < -88.0f ? 0.0f : tr_sigmoid(g);
        a = g * s;
        da = fmaf(a, 1.0f - s, s);
        if (g < -88.0f) a = da = 0.0f;
    } else {
        const float phi = 0.5f * erfcf(-0.70710678118654752f * g);
        a = g * phi;
        da = fmaf(g * 0.3989422804014327f, __expf(-0.5f * g * g), phi);
    }
}

__device__ __forceinline__ void tr_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void tr_store(__half* p, float v) { *p = __float2half_rn(v); }

}  // namespace evo
