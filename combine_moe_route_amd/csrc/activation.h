// Activations shared by the bf16 grouped GEMM's epilogue and the gated
// activation between the FP8 products. fp32 throughout.
#pragma once

#include "moe_device.h"

namespace moe {

enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == kActRelu) return z < 0.0f ? 0.0f : z;      // NaN stays NaN
    // z * sigmoid(z): exp(-z) overflows to inf for very negative z, giving -0
    if constexpr (ACT == kActSilu) return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
    // erfc keeps the relative precision of the negative tail, 1 + erf does not
    if constexpr (ACT == kActGelu) return 0.5f * z * erfcf(z * -0.70710678118654752f);
    return z;
}

// Two fp32 values to two bf16 (nearest even, NaN kept), one instruction.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

}  // namespace moe
