// Activations of the fused linear layer and their slopes, in fp32.
//
// Results are rounded to bf16 (half a step is 2^-8 of the value), so exp
// through the fast base-2 exponential and division through the fast
// reciprocal (together within 2^-17 relative for |x| < 88; beyond, results
// below 10^-36 become zero) are exact enough.  The forms are chosen so that
// nothing cancels for negative arguments, where x (1 + erf) or x (1 + tanh)
// would.
#pragma once

#include <math.h>

#include "qkn_common.cuh"

namespace qkn {
namespace lin {

// 1 / (1 + e^-x)
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// The normal distribution function Phi(z) and e^(-z^2 / 2).  For a = |z|
//   Phi(-a) = e^(-a^2 / 2) t P(t),  t = 1 / (1 + 0.36 a)
// with P the degree-6 polynomial of least relative error on 0 <= a <= 14
// (weighted least squares against erfcx, 2^-20; 2^-18 in fp32), and
// Phi(a) = 1 - Phi(-a): the relative error stays small in the left tail,
// where 1 + erf(z / sqrt 2) has none of its digits left.  About 15
// instructions; erfcf's 70 made the epilogue of a 256 x 256 tile as long as
// the products of 2048 k.
__device__ __forceinline__ float normal_cdf(float z, float &gauss) {
    const float a = fabsf(z), t = __fdividef(1.f, fmaf(0.36f, a, 1.f));
    gauss = __expf(-0.5f * z * z);
    float p = fmaf(0.04705606773495674f, t, -0.17976394295692444f);
    p = fmaf(p, t, 0.1809530258178711f);
    p = fmaf(p, t, 0.026549967005848885f);
    p = fmaf(p, t, 0.13971905410289764f);
    p = fmaf(p, t, 0.14177249372005463f);
    p = fmaf(p, t, 0.14371304214000702f);
    const float q = p * t * gauss;
    return z < 0.f ? q : 1.f - q;
}

constexpr float kTanhA = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

template <int ACT> __device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == QKN_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN stays
    if constexpr (ACT == QKN_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
    if constexpr (ACT == QKN_ACT_GELU) {
        float gauss;
        return z * normal_cdf(z, gauss);
    }
    if constexpr (ACT == QKN_ACT_GELU_TANH)  // 0.5 z (1 + tanh u) = z / (1 + e^-2u)
        return __fdividef(z, 1.f + __expf(-kTanhA * (z + kTanhB * z * z * z)));
    return z;
}

__device__ __forceinline__ float slope(int act, float z) {
    switch (act) {
    case QKN_ACT_RELU:
        return z > 0.f ? 1.f : z <= 0.f ? 0.f : z;  // NaN stays
    case QKN_ACT_SILU: {
        const float p = sigmoid(z);
        return p * (1.f + z * (1.f - p));
    }
    case QKN_ACT_GELU: {
        float gauss;
        const float cdf = normal_cdf(z, gauss);
        return cdf + z * (0.39894228040143268f * gauss);
    }
    case QKN_ACT_GELU_TANH: {
        const float p = sigmoid(kTanhA * (z + kTanhB * z * z * z));
        return p + z * p * (1.f - p) * kTanhA * (1.f + 3.f * kTanhB * z * z);
    }
    default:
        return 1.f;
    }
}

// What the epilogues add to the product.
struct Epilogue {
    const float *inv_rms;  // [M] row scale, or null
    const void *bias;      // [N], or null
    int bias_bf16;
};

// Bias of 8 columns (16-byte aligned), 0 without one.
__device__ __forceinline__ void load_bias8(const Epilogue &e, int col, float (&b)[8]) {
    if (e.bias == nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = 0.f;
    } else if (e.bias_bf16) {
        load_weights_batched<__nv_bfloat16, 8>(static_cast<const __nv_bfloat16 *>(e.bias) + col, b);
    } else {
        load_weights_batched<float, 8>(static_cast<const float *>(e.bias) + col, b);
    }
}

}  // namespace lin
}  // namespace qkn
