// Gated activation between the two FP8 grouped GEMMs: for every row of the
// dispatch segments
//   v[c] = act(h[c]) * h[I + c]                       (fp32)
//   s    = max |v| over 128 channels / 448            (fp32)
//   code = E4M3(v / s), nearest even, saturated; s == 0 gives zero codes
// the same quantisation as the FP8 dispatch. Bound by memory: 4 I bytes read
// and I + I / 32 written a row.
//
// 16 lanes own one block of 128 channels (8 channels, two 16-byte loads and
// one 8-byte store each); the block's maximum is a DPP butterfly.
#include "activation.h"
#include "launch.h"

namespace moe {

namespace {

constexpr int kGatedThreads = 256;

template <int ACT>
__global__ __launch_bounds__(kGatedThreads) void k_gated_act_fp8(
    const uint16_t* __restrict__ h, const int32_t* __restrict__ expert_offsets, int E,
    int64_t max_rows, int I, uint8_t* __restrict__ out, float* __restrict__ out_scales) {
    int64_t used = expert_offsets[E];
    used = used < max_rows ? used : max_rows;
    const int nb = I / 128;
    const int64_t units = used * nb;
    const int sub = threadIdx.x & 15;
    for (int64_t u = ((int64_t)blockIdx.x * kGatedThreads + threadIdx.x) >> 4; u < units;
         u += (int64_t)gridDim.x * (kGatedThreads / 16)) {
        const int64_t r = u / nb;
        const int b = (int)(u - r * nb);
        const uint16_t* row = h + r * 2 * I + b * 128 + sub * 8;
        float g[8], v[8];
        unpack8(*reinterpret_cast<const uint4*>(row), g);
        unpack8(*reinterpret_cast<const uint4*>(row + I), v);
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            v[i] *= activate<ACT>(g[i]);
            amax = fmaxf(amax, fabsf(v[i]));
        }
        amax = group8_max(amax);
        amax = fmaxf(amax, dpp_f32<kDppRowMirror>(amax));
        const float s = amax / 448.0f;
        uint2 q = make_uint2(0u, 0u);
        if (s != 0.0f) {
            q.x = f32x4_to_e4m3(v[0] / s, v[1] / s, v[2] / s, v[3] / s);
            q.y = f32x4_to_e4m3(v[4] / s, v[5] / s, v[6] / s, v[7] / s);
        }
        *reinterpret_cast<uint2*>(out + r * I + b * 128 + sub * 8) = q;
        if (sub == 0) out_scales[u] = s;
    }
}

}  // namespace

hipError_t launch_gated_act_fp8(const void* h, const int32_t* expert_offsets, int E,
                                int64_t max_rows, int I, int act, void* out, float* out_scales,
                                hipStream_t stream, LaunchInfo* info, bool run) {
    const int64_t units = max_rows * (I / 128);
    const int64_t need = (units + kGatedThreads / 16 - 1) / (kGatedThreads / 16);
    const int64_t blocks = need < 2048 ? need : 2048;
    if (info) *info = LaunchInfo{blocks, kGatedThreads, 0, act, "gated_act_fp8"};
    if (!run || blocks == 0) return hipSuccess;
    const dim3 grid((unsigned)blocks), block(kGatedThreads);
    const auto* h16 = static_cast<const uint16_t*>(h);
    auto* o8 = static_cast<uint8_t*>(out);
    switch (act) {
        case kActRelu:
            k_gated_act_fp8<kActRelu><<<grid, block, 0, stream>>>(h16, expert_offsets, E, max_rows,
                                                                  I, o8, out_scales);
            break;
        case kActSilu:
            k_gated_act_fp8<kActSilu><<<grid, block, 0, stream>>>(h16, expert_offsets, E, max_rows,
                                                                  I, o8, out_scales);
            break;
        case kActGelu:
            k_gated_act_fp8<kActGelu><<<grid, block, 0, stream>>>(h16, expert_offsets, E, max_rows,
                                                                  I, o8, out_scales);
            break;
        default:
            k_gated_act_fp8<kActNone><<<grid, block, 0, stream>>>(h16, expert_offsets, E, max_rows,
                                                                  I, o8, out_scales);
    }
    return hipGetLastError();
}

}  // namespace moe
