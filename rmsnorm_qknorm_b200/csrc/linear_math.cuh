// Activations of the fused linear layer and their slopes, in fp32.
//
// Results are rounded to bf16 (half a step is 2^-8 of the value), so the fast
// base-2 exponential and reciprocal are exact enough (together within 2^-17
// relative for |x| < 88; beyond, results below 10^-36 become zero).  The
// forms are chosen so that nothing cancels for negative arguments, where
// x (1 + erf) or x (1 + tanh) would.  Two values at a time: products and sums
// take the packed fp32x2 instructions, which round like scalar ones.
#pragma once

#include <math.h>

#include "qkn_common.cuh"

namespace qkn {
namespace lin {

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float relu(float x) {  // NaN stays
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 pair_of(float v) { return make_float2(v, v); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhA = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

// 1 / (1 + 2^u)
__device__ __forceinline__ float2 logistic2(float2 u) {
    const float2 d = __fadd2_rn(make_float2(exp2_fast(u.x), exp2_fast(u.y)), pair_of(1.f));
    return make_float2(rcp_fast(d.x), rcp_fast(d.y));
}

// The normal distribution's left tail Phi(-a), and gauss = e^(-a^2 / 2), for a >= 0:
//   Phi(-a) = e^(-a^2 / 2) t P(t),  t = 1 / (1 + 0.36 a)
// with P the degree-6 polynomial of least relative error on 0 <= a <= 14
// (weighted least squares against erfcx, 2^-20; 2^-17 in fp32).
__device__ __forceinline__ float2 normal_tail2(float2 a, float2 &gauss) {
    const float2 d = __ffma2_rn(a, pair_of(0.36f), pair_of(1.f));
    const float2 t = make_float2(rcp_fast(d.x), rcp_fast(d.y));
    const float2 u = __fmul2_rn(__fmul2_rn(a, a), pair_of(-0.5f * kLog2e));
    gauss = make_float2(exp2_fast(u.x), exp2_fast(u.y));
    float2 p = __ffma2_rn(t, pair_of(0.04705606773495674f), pair_of(-0.17976394295692444f));
    p = __ffma2_rn(p, t, pair_of(0.1809530258178711f));
    p = __ffma2_rn(p, t, pair_of(0.026549967005848885f));
    p = __ffma2_rn(p, t, pair_of(0.13971905410289764f));
    p = __ffma2_rn(p, t, pair_of(0.14177249372005463f));
    p = __ffma2_rn(p, t, pair_of(0.14371304214000702f));
    return __fmul2_rn(__fmul2_rn(p, t), gauss);
}

template <int ACT> __device__ __forceinline__ float2 activate2(float2 z) {
    if constexpr (ACT == QKN_ACT_RELU) return make_float2(relu(z.x), relu(z.y));
    if constexpr (ACT == QKN_ACT_SILU) return __fmul2_rn(z, logistic2(__fmul2_rn(z, pair_of(-kLog2e))));
    if constexpr (ACT == QKN_ACT_GELU) {
        // z Phi(z) = max(z, 0) - |z| Phi(-|z|) on either side; |z| is cut where its term is zero,
        // so that infinities do not meet that zero
        const float2 a = make_float2(fminf(fabsf(z.x), 1e4f), fminf(fabsf(z.y), 1e4f));
        float2 gauss;
        const float2 q = __fmul2_rn(normal_tail2(a, gauss), pair_of(-1.f));
        return __ffma2_rn(a, q, make_float2(relu(z.x), relu(z.y)));
    }
    if constexpr (ACT == QKN_ACT_GELU_TANH) {  // 0.5 z (1 + tanh u) = z / (1 + e^-2u)
        const float2 w = __ffma2_rn(__fmul2_rn(z, z), pair_of(-kLog2e * kTanhA * kTanhB), pair_of(-kLog2e * kTanhA));
        return __fmul2_rn(z, logistic2(__fmul2_rn(z, w)));
    }
    return z;
}

// act'(z)
template <int ACT> __device__ __forceinline__ float2 slope2(float2 z) {
    if constexpr (ACT == QKN_ACT_RELU)  // NaN stays
        return make_float2(z.x > 0.f ? 1.f : z.x <= 0.f ? 0.f : z.x, z.y > 0.f ? 1.f : z.y <= 0.f ? 0.f : z.y);
    if constexpr (ACT == QKN_ACT_SILU) {  // p (1 + z (1 - p)) = p + z p (1 - p)
        const float2 p = logistic2(__fmul2_rn(z, pair_of(-kLog2e)));
        const float2 r = __ffma2_rn(p, pair_of(-1.f), pair_of(1.f));
        return __fmul2_rn(p, __ffma2_rn(z, r, pair_of(1.f)));
    }
    if constexpr (ACT == QKN_ACT_GELU) {  // Phi(z) + z phi(z)
        const float2 a = make_float2(fminf(fabsf(z.x), 1e4f), fminf(fabsf(z.y), 1e4f));
        float2 gauss;
        const float2 q = normal_tail2(a, gauss);
        const float2 cdf = make_float2(z.x < 0.f ? q.x : 1.f - q.x, z.y < 0.f ? q.y : 1.f - q.y);
        return __ffma2_rn(z, __fmul2_rn(gauss, pair_of(0.39894228040143268f)), cdf);
    }
    if constexpr (ACT == QKN_ACT_GELU_TANH) {
        // z^2 is cut where p (1 - p) has long been zero, so that its overflow (|z| above 1.8e19) does not meet that zero
        const float2 sq = __fmul2_rn(z, z), zz = make_float2(fminf(sq.x, 1e8f), fminf(sq.y, 1e8f));
        const float2 w = __ffma2_rn(zz, pair_of(-kLog2e * kTanhA * kTanhB), pair_of(-kLog2e * kTanhA));
        const float2 p = logistic2(__fmul2_rn(z, w));
        const float2 r = __ffma2_rn(p, pair_of(-1.f), pair_of(1.f));
        const float2 d = __ffma2_rn(zz, pair_of(3.f * kTanhA * kTanhB), pair_of(kTanhA));  // (2 u)'
        return __ffma2_rn(__fmul2_rn(z, __fmul2_rn(p, r)), d, p);
    }
    return pair_of(1.f);
}

// What the epilogues add to the product.
struct Epilogue {
    const float *inv_rms;  // [M] row scale, or null
    const void *bias;      // [N], or null
    int bias_bf16;
};

}  // namespace lin
}  // namespace qkn
