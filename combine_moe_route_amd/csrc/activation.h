// Activations of the bf16 and INT8 grouped GEMMs' epilogue and of the gated activations
// between two products (FP8, INT8), in fp32 throughout; and the rounding to bf16 that
// these and the quantising norm share.
#pragma once

#include "moe_device.h"

namespace moe {

enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };

// z Phi(z), Phi the normal distribution: for z < 0 it is z h, else z (1 - h), with
// h = erfc(x) / 2, x = |z| / sqrt 2. erfc(x) = t Q(t) exp(-x^2), t = 1 / (1 + 0.3 x),
// where Q is the polynomial of degree 8 fitted to exp(x^2) erfc(x) / t over
// 0 <= x <= 12; with its coefficients in fp32 it is off by at most 5.7e-8 of the
// value. In fp32 the result is within 2^-21 |z|. Relatively it is within 1e-6 down
// to z = -4, 3e-6 to -8 and 8e-6 to -13 (the exponent's roundings grow with z^2);
// below -13.2 the exponential is under 2^-126 and may count as 0. The device
// library's erfc took four times the instructions: with it the gated activation of
// 6185 rows of 1408 channels was bound by them.
__device__ __forceinline__ float gelu_poly(float t) {
    float q = -0.129252457f;
    q = fmaf(q, t, 0.484298284f);
    q = fmaf(q, t, -0.509765798f);
    q = fmaf(q, t, 0.544960012f);
    q = fmaf(q, t, -0.0928216458f);
    q = fmaf(q, t, 0.214179706f);
    q = fmaf(q, t, 0.148521657f);
    q = fmaf(q, t, 0.170690877f);
    return fmaf(q, t, 0.169189357f);
}

__device__ __forceinline__ float gelu(float z) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.21213203435596426f, fabsf(z), 1.0f));
    const float h = 0.5f * t * gelu_poly(t) * __expf(-0.5f * z * z);
    // from z = 14 on h is 0, so 16 stands for any larger z: inf times 0 would be NaN
    return z < 0.0f ? z * h : fmaf(-fminf(z, 16.0f), h, z);
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == kActRelu) return z < 0.0f ? 0.0f : z;      // NaN stays NaN
    // z * sigmoid(z): exp(-z) overflows to inf for very negative z, giving -0
    if constexpr (ACT == kActSilu) return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
    if constexpr (ACT == kActGelu) return gelu(z);
    return z;
}

// Two fp32 values to two bf16 (nearest even, NaN kept), one instruction.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

}  // namespace moe
