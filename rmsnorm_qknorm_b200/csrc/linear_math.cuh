// Activations of the fused linear layer and their slopes, in fp32.
//
// Results are rounded to bf16 (half a step is 2^-9 relative), so exp through
// the fast base-2 exponential (relative error below 2^-17 for |x| < 88, where
// it saturates) is exact enough; the forms are chosen so that nothing cancels
// for negative arguments, where x * (1 + erf) or x * (1 + tanh) would.
#pragma once

#include <math.h>

#include "qkn_common.cuh"

namespace qkn {
namespace lin {

// 1 / (1 + e^-x)
__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + __expf(-x)); }

constexpr float kTanhA = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

template <int ACT> __device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == QKN_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN stays
    if constexpr (ACT == QKN_ACT_SILU) return z / (1.f + __expf(-z));
    if constexpr (ACT == QKN_ACT_GELU) return 0.5f * z * erfcf(-0.70710678118654752f * z);
    if constexpr (ACT == QKN_ACT_GELU_TANH)  // 0.5 z (1 + tanh u) = z / (1 + e^-2u)
        return z / (1.f + __expf(-kTanhA * (z + kTanhB * z * z * z)));
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
    case QKN_ACT_GELU:
        return 0.5f * erfcf(-0.70710678118654752f * z) + z * (0.39894228040143268f * __expf(-0.5f * z * z));
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
    int has_res, has_z;
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
