// Gated activation between the two FP8 grouped GEMMs: for every row of the
// dispatch segments
//   v[c] = act(h[c]) * h[I + c]                       (fp32)
//   s    = max |v| over 128 channels / 448            (fp32)
//   code = E4M3(v / s), nearest even, saturated; s == 0 gives zero codes
// (v past fp32's range counts as the largest finite value), the same
// quantisation as the FP8 dispatch. 4 I bytes read and I + I / 32 written a row:
// 147 thousand rows of 2048 channels (1.51 GB) 243 us, 6.2 TB/s. There memory and
// instructions are both near their limits (counters: 27.5 vector instructions a
// value with SiLU, which at four cycles each fill 97 % of the cycles); GELU with
// 6185 rows of 1408 is bound by instructions (96 %).
//
// 16 lanes own one block of 128 channels (8 channels, two 16-byte loads and one
// 8-byte store each); the block's maximum is a DPP butterfly. A lane has up to
// two blocks in hand at a time, all loads first (262 us; four: 272 us). Loads
// and stores carry the non-temporal hint (plain loads 283 against 272 us, plain
// stores 272 against 256 us, each with four blocks in hand).
//
// The quotient is v * (1 / s) with one correction, q += (v - q s) (1 / s): with
// a correctly rounded reciprocal the corrected q is the correctly rounded v / s
// (Markstein) as long as the residual is exact, which s >= 2^-100 ensures;
// below that the division itself is used. Three instructions instead of about
// ten: with eight divisions a lane the kernel was bound by instructions.
#include "activation.h"
#include "launch.h"

namespace moe {

namespace {

constexpr int kGatedThreads = 256;
constexpr int kUnits = kGatedThreads / 16;   // 128-channel blocks a workgroup takes at a time
constexpr int kDepth = 2;                    // blocks of a lane in flight
constexpr float kMaxFloat = 0x1.fffffep127f; // largest finite fp32

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// act(g) * u for bf16 g and u, as close as fp32 steps come (an error of v moves
// the codes that lie at a rounding border). g u is exact in fp32, so the gate's
// factor is multiplied in last. The arguments of the exponentials are exact too:
// log2 e is split so that its upper part times a bf16 value fits fp32, or the
// product's rounding error is kept, and the rest corrects the result to first
// order; the reciprocals get a Newton step. Of 33 million codes 31 to 49 then
// differ from those of 64-bit arithmetic with silu and 39 to 60 with gelu (the
// rounding of s alone moves most of them); fp32 with the library's exp, erf and
// divisions 32 to 51 and 64 to 93.
template <int ACT>
__device__ __forceinline__ float gated_product(float g, float u) {
    const float p = g * u;
    if constexpr (ACT == kActRelu) return g < 0.0f ? 0.0f : p;
    if constexpr (ACT == kActSilu) {
        float e = __builtin_amdgcn_exp2f(-1.44268798828125f * g);
        e = fmaf(e, -4.88849515e-06f * g, e);            // (log2 e - the above) ln 2
        const float d = 1.0f + e;
        float r = __builtin_amdgcn_rcpf(d);
        r = fmaf(fmaf(-d, r, 1.0f), r, r);
        // d is inf for g below -88.7; it stays NaN for a NaN gate. A reciprocal below
        // 2^-126 (g below -87.3) may count as 0.
        return d == INFINITY ? 0.0f : p * r;
    }
    if constexpr (ACT == kActGelu) {
        const float d = fmaf(0.21213203435596426f, fabsf(g), 1.0f);
        float t = __builtin_amdgcn_rcpf(d);
        t = fmaf(fmaf(-d, t, 1.0f), t, t);
        const float y = fmaxf(-0.5f * g * g, -200.0f);   // exp(-200) is 0
        const float a = 1.44269504f * y;
        const float rest = fmaf(y, 1.92596299e-08f, fmaf(y, 1.44269504f, -a));
        float e = __builtin_amdgcn_exp2f(a);
        e = fmaf(e, 0.693147181f * rest, e);
        const float h = 0.5f * t * gelu_poly(t) * e;
        return g < 0.0f ? p * h : fmaf(-p, h, p);
    }
    return p;
}

template <int ACT>
__global__ __launch_bounds__(kGatedThreads) void k_gated_act_fp8(
    const uint16_t* __restrict__ h, const int32_t* __restrict__ expert_offsets, int E,
    int64_t max_rows, int I, int rows, uint32_t magic, uint8_t* __restrict__ out,
    float* __restrict__ out_scales) {
    const int64_t end = expert_offsets[E];
    const int64_t used = end < max_rows ? end : max_rows;
    const int64_t r0 = (int64_t)blockIdx.x * rows;
    if (r0 >= used) return;
    const int nb = I / 128;
    const int n = (int)(used - r0 < rows ? used - r0 : rows) * nb;
    const int sub = threadIdx.x & 15;
    const uint16_t* const base = h + r0 * 2 * I;
    for (int u0 = threadIdx.x >> 4; u0 < n; u0 += kUnits * kDepth) {
        u32x4 g4[kDepth], u4[kDepth];
#pragma unroll
        for (int d = 0; d < kDepth; d++) {
            const int u = u0 + d * kUnits;
            if (u < n) {
                // row u / nb, exact by the launcher's magic number
                const int row = magic ? (int)__umulhi((uint32_t)u, magic) : u;
                const uint16_t* at = base + (int64_t)(u + row * nb) * 128 + sub * 8;
                g4[d] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(at));
                u4[d] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(at + I));
            }
        }
#pragma unroll
        for (int d = 0; d < kDepth; d++) {
            const int u = u0 + d * kUnits;
            if (u >= n) break;
            float g[8], v[8], amax = 0.0f;
            unpack8(make_uint4(g4[d][0], g4[d][1], g4[d][2], g4[d][3]), g);
            unpack8(make_uint4(u4[d][0], u4[d][1], u4[d][2], u4[d][3]), v);
            float pmax = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                pmax = fmaxf(pmax, fabsf(g[i] * v[i]));
                v[i] = gated_product<ACT>(g[i], v[i]);
                amax = fmaxf(amax, fabsf(v[i]));
            }
            // g u out of range: act(g) u maybe not. If it is, the largest finite value
            // stands for it (|act(g)| <= |g|, so only here): an infinite v or s would
            // make NaN of the whole block below.
            if (!(pmax < INFINITY)) {
                amax = 0.0f;
                unpack8(make_uint4(u4[d][0], u4[d][1], u4[d][2], u4[d][3]), v);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    v[i] *= activate<ACT>(g[i]);
                    v[i] = v[i] > kMaxFloat ? kMaxFloat : v[i] < -kMaxFloat ? -kMaxFloat : v[i];
                    amax = fmaxf(amax, fabsf(v[i]));
                }
            }
            amax = group8_max(amax);
            amax = fmaxf(amax, dpp_f32<kDppRowMirror>(amax));
            const float s = amax / 448.0f;
            float q[8];
            u32x2 code;
            if (s >= 0x1p-100f) {
                // |q| <= 448 (1 + 2^-22) rounds to at most 448: no clamp
                const float inv = 1.0f / s;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    q[i] = v[i] * inv;
                    q[i] = fmaf(fmaf(-q[i], s, v[i]), inv, q[i]);
                }
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    int c = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * x], q[4 * x + 1], 0, false);
                    c = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * x + 2], q[4 * x + 3], c, true);
                    code[x] = (uint32_t)c;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) q[i] = s > 0.0f ? v[i] / s : 0.0f;
                code = {f32x4_to_e4m3(q[0], q[1], q[2], q[3]),
                        f32x4_to_e4m3(q[4], q[5], q[6], q[7])};
            }
            __builtin_nontemporal_store(
                code, reinterpret_cast<u32x2*>(out + r0 * I + (int64_t)u * 128 + sub * 8));
            if (sub == 0) out_scales[r0 * nb + u] = s;
        }
    }
}

}  // namespace

hipError_t launch_gated_act_fp8(const void* h, const int32_t* expert_offsets, int E,
                                int64_t max_rows, int I, int act, void* out, float* out_scales,
                                hipStream_t stream, LaunchInfo* info, bool run) {
    // rows per workgroup: about kDepth blocks of 128 channels per 16 lanes.
    // magic = ceil(2^32 / nb): u * magic >> 32 is u / nb for u nb < 2^32, and
    // u < rows nb is at most 2^13 here. One block a row: 0, no division.
    const int nb = I / 128;
    const int rows = nb < kUnits * kDepth ? kUnits * kDepth / nb : 1;
    const uint32_t magic = (uint32_t)((((uint64_t)1 << 32) + nb - 1) / nb);   // 2^32 wraps to 0
    const int64_t blocks = (max_rows + rows - 1) / rows;
    if (info) *info = LaunchInfo{blocks, kGatedThreads, 0, act, "gated_act_fp8"};
    if (!run || blocks == 0) return hipSuccess;
    const dim3 grid((unsigned)blocks), block(kGatedThreads);
    const auto* h16 = static_cast<const uint16_t*>(h);
    auto* o8 = static_cast<uint8_t*>(out);
    auto launch = [&](auto kernel) {
        kernel<<<grid, block, 0, stream>>>(h16, expert_offsets, E, max_rows, I, rows, magic, o8,
                                           out_scales);
    };
    switch (act) {
        case kActRelu: launch(k_gated_act_fp8<kActRelu>); break;
        case kActSilu: launch(k_gated_act_fp8<kActSilu>); break;
        case kActGelu: launch(k_gated_act_fp8<kActGelu>); break;
        default: launch(k_gated_act_fp8<kActNone>);
    }
    return hipGetLastError();
}

}  // namespace moe
