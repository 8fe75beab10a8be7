// The gate's activations and the power-of-two exponents that the products through packed weights
// share between their kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "awq_internal.h"

namespace awq {

// Power-of-two exponent k with max * 2^-k in [2^(top-1), 2^top) (0 for a zero or non-finite
// max), clamped to [-125, 125] so that 2^k and 2^-k stay normal floats.
__device__ __forceinline__ int scale_exp(float mx, int top) {
    if (!(mx > 0.0f) || isinf(mx)) return 0;
    int e;
    frexpf(mx, &e);                                    // mx = f * 2^e, f in [0.5, 1)
    const int k = e - top;
    return k < -125 ? -125 : (k > 125 ? 125 : k);
}

// The layer's exponent kW: dequantised weights are held as (code - z) * Delta * 2^-kW, with
// 15 * max |Delta| * 2^-kW < 2^15, so they stay in fp16's normal range whatever the layer's
// magnitude.  dmax holds the maxima of DMAX_PARTS parts of the scales as fp16 bits (those of
// non-negative values order as the values).  A converged warp's collective.
// (Read through L1: from L2 alone, the many blocks of a dequantisation lost 25 us to these lines.)
__device__ __forceinline__ int dq_exp(const unsigned *dmax) {
    const uint4 v = reinterpret_cast<const uint4 *>(dmax)[threadIdx.x & 31];
    const unsigned mb = __reduce_max_sync(0xffffffffu, max(max(v.x, v.y), max(v.z, v.w)));
    return scale_exp(__half2float(__ushort_as_half(static_cast<unsigned short>(mb))), 11);
}
__device__ __forceinline__ float dq_scale(const unsigned *dmax) { return ldexpf(1.0f, dq_exp(dmax)); }

// The exponent e that a token's gate and up gradients are divided by (as 2^e) before they are
// rounded to fp16.  grow bounds max |dh| * ||x / s|| < 2^grow (DGU_NONE: zero or not finite);
// every |g|, |u| is at most ||x / s|| * ||W_o|| <= ||x / s|| * sqrt(inner) * 15 max |Delta|
// (Cauchy-Schwarz), |act(g)| <= |g|, |act'| < 1.2, so the scaled values are below 2^15.  The bound is
// typically 2^8 above the largest value, which leaves fp16's normal range 20 binades below that.
constexpr int DGU_NONE = -100000;
__device__ __forceinline__ int dgu_exp(int grow, int inner, int kw) {
    if (grow <= DGU_NONE) return 0;
    int r;
    frexpf(sqrtf(static_cast<float>(inner)) * 1.2f, &r);
    const int k = grow + r + (kw + 15) - 15;           // 15 max |Delta| < 2^(kW + 15)
    return k < -125 ? -125 : (k > 125 ? 125 : k);
}

// What rounding to bf16 takes off v (exact; 0 where v or its rounding is not finite, so that an infinite gradient stays
// infinite).
__device__ __forceinline__ float bf16_rest(float v) {
    const float r = v - __bfloat162float(__float2bfloat16_rn(v));
    return fabsf(r) < INFINITY ? r : 0.0f;
}

// (2 ulp; exp(-g) = inf below about -88 gives 0)
__device__ __forceinline__ float act_sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// act(g) and its derivative:
//   SiLU        g sig(g);                 sig (1 + g (1 - sig))
//   GELU        g Phi(g);                 Phi + g phi
//   GELU, tanh  g (1 + tanh v) / 2, v = sqrt(2/pi) (g + 0.044715 g^3)
// SiLU is written with g only as a factor of a bounded term; for g below about -88 exp(-g) is
// inf and the quotient 0, as it should be.
__device__ __forceinline__ float act_both(float g, int act, float &d) {
    if (act == ACT_SILU) {
        const float s = act_sigmoid(g);
        d = s * (1.0f + g * (1.0f - s));
        return g * s;
    }
    if (act == ACT_GELU) {
        const float cdf = 0.5f * erfcf(g * -0.70710678118654752f);
        d = cdf + g * (0.3989422804014327f * __expf(-0.5f * g * g));
        return g * cdf;
    }
    const float c = 0.7978845608028654f;
    // (1 + tanh v) / 2 = sig(2 v)
    const float s = act_sigmoid(2.0f * c * g * (1.0f + 0.044715f * g * g));
    // s (1 - s) is 0 in fp32 from |g| = 16 on (exp(-300)), where g's powers, from 2^64 on infinite, would make it NaN
    const float b = fminf(fmaxf(g, -16.0f), 16.0f);
    d = s + b * (2.0f * s * (1.0f - s)) * c * (1.0f + 3.0f * 0.044715f * b * b);
    return g * s;
}
__device__ __forceinline__ float act_value(float g, int act) {
    float d;
    return act_both(g, act, d);
}

}  // namespace awq
