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

// sigmoid(g) from e^-|g| <= 1, which cannot overflow and goes to 0 with e^g on the
// negative side.  expf's error is an ulp or so (__expf's grows with |g|, to 100 ulp at
// g = -85, and all of it would reach act(g) there); __fdividef is within 2 ulp for
// denominators as here, from 1 to 2.
__device__ __forceinline__ float tr_sigmoid(float g) {
    const float e = expf(-fabsf(g));
    return __fdividef(g < 0.0f ? e : 1.0f, 1.0f + e);
}

// A gate as a factor of its sigmoid or Phi: above -infinity, so that a sum G that has
// overflowed gives act's limit 0 and not 0 times infinity.  NaN stays.
__device__ __forceinline__ float tr_above(float g) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(g) : "f"(-3.402823466e38f));
    return g;
}
// The same on both sides, for the term of act' that vanishes on both.
__device__ __forceinline__ float tr_finite(float g) {
    g = tr_above(g);
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(g) : "f"(3.402823466e38f));
    return g;
}

// act(g) and its derivative.  silu: g s, s + g s (1 - s) with s = sigmoid(g);
// gelu: g Phi(g), Phi(g) + g phi(g), Phi and phi the normal distribution and density.
template <int ACT>
__device__ __forceinline__ float tr_act(float g) {
    if constexpr (ACT == EVO_ACT_SILU) return tr_above(g) * tr_sigmoid(g);
    else return tr_above(g) * (0.5f * erfcf(-0.70710678118654752f * g));
}

template <int ACT>
__device__ __forceinline__ void tr_act_grad(float g, float& a, float& da) {
    if constexpr (ACT == EVO_ACT_SILU) {
        const float s = tr_sigmoid(g);
        a = tr_above(g) * s;
        da = fmaf(tr_finite(g) * s, 1.0f - s, s);
    } else {
        const float phi = 0.5f * erfcf(-0.70710678118654752f * g);
        a = tr_above(g) * phi;
        da = fmaf(tr_finite(g) * 0.3989422804014327f, expf(-0.5f * g * g), phi);
    }
}

__device__ __forceinline__ void tr_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void tr_store(__half* p, float v) { *p = __float2half_rn(v); }

}  // namespace evo
