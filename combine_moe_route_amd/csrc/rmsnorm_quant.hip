// The norm in front of an expert layer: the residual's addition, the
// root-mean-square norm, and an output in 8 bits with scales (and, for the gate,
// one in bf16). For every token, in fp32:
//
//   h = x + residual                       sum = bf16(h), the next residual
//   v = h w / sqrt(mean(h^2) + eps)        y   = bf16(v)
//   int8  s = max |v| / 127 over the token,          code = 127 v / max |v|
//   fp8   s = max |v| / 448 over 128 channels,       code = 448 v / max |v|
//
// The norm's factor r is common to a token, so codes are formed from h w alone:
// 127 h w / max |h w|. With bf16 inputs h w has few more bits than fp32 (without a
// residual 16, exactly), and the quotient is formed with a factor in two parts, so
// a code differs from that of exact arithmetic only where the value lies within
// about 2^-24 of a border.
//
// Squares leave fp32's range where |h| nears 2^64: such a token (its sum of
// squares is not finite) is done again with h divided by the power of two of its
// largest |h|, which is exact for what counts. If the sum is still not finite the
// token holds an infinity or NaN: y is NaN, the codes are 0 and its scales NaN, so
// that what it is multiplied into is NaN and no other token notices.
//
// One pass: a token's row stays in registers (C pieces of 8 channels a lane). Past H =
// 32768 the eight pieces need more than the 128 that a workgroup of 1024 threads leaves a
// lane, and 45 (int8) or 12 (fp8) spill: 4096 tokens of 65536, residual and all outputs,
// 4.2 and 5.2 TB/s, of 32768 5.5.
#include "activation.h"
#include "launch.h"

#include <type_traits>

namespace moe {

namespace {

constexpr float kInf = __builtin_inff();

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ u32x4 load_nt(const uint16_t* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}

// Eight values times r as bf16.
__device__ __forceinline__ uint4 bf16x8_of(const float* f, float r) {
    return make_uint4(cvt_bf16x2(f[0] * r, f[1] * r), cvt_bf16x2(f[2] * r, f[3] * r),
                      cvt_bf16x2(f[4] * r, f[5] * r), cvt_bf16x2(f[6] * r, f[7] * r));
}

struct FMax {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
};

__device__ __forceinline__ float wave_sum(float v) {
    return __uint_as_float(group_reduce<kWave>(__float_as_uint(v), FAdd()));
}
__device__ __forceinline__ float wave_max(float v) {
    return __uint_as_float(group_reduce<kWave>(__float_as_uint(v), FMax()));
}

// Sum and maximum over the threads of a row: a wave, or the whole workgroup.
template <bool WAVE_ROW>
__device__ __forceinline__ void reduce_row(float& sum, float& top, float2* lds) {
    sum = wave_sum(sum);
    top = wave_max(top);
    if constexpr (!WAVE_ROW) {
        const int waves = blockDim.x / kWave;
        if ((threadIdx.x & (kWave - 1)) == 0) lds[threadIdx.x / kWave] = make_float2(sum, top);
        __syncthreads();
        sum = top = 0.0f;
        for (int w = 0; w < waves; w++) {
            sum += lds[w].x;
            top = fmaxf(top, lds[w].y);
        }
        __syncthreads();                       // the row may be reduced again
    }
}

template <bool FP8, int C, bool WAVE_ROW>
__global__ __launch_bounds__(WAVE_ROW ? 256 : 1024) void k_rmsnorm_quant(NormArgs a) {
    __shared__ float2 lds[1024 / kWave];
    const int64_t t = WAVE_ROW ? (int64_t)blockIdx.x * 4 + threadIdx.x / kWave : blockIdx.x;
    if (t >= a.T) return;
    const int tid = WAVE_ROW ? threadIdx.x & (kWave - 1) : threadIdx.x;
    const int nt = WAVE_ROW ? kWave : blockDim.x;
    const int U = a.H / 8;
    const int64_t at = t * a.H;
    u32x4 xv[C], rv[C], wv[C];
#pragma unroll
    for (int i = 0; i < C; i++) {
        const int u = tid + i * nt;
        xv[i] = rv[i] = wv[i] = u32x4{0u, 0u, 0u, 0u};
        if (u < U) {
            xv[i] = load_nt(a.x + t * a.ld + 8 * u);
            if (a.residual) rv[i] = load_nt(a.residual + at + 8 * u);
            wv[i] = *reinterpret_cast<const u32x4*>(a.weight + 8 * u);
        }
    }
    float h[C][8], sum = 0.0f, top = 0.0f;
    auto weight = [&](int i, float* w) {
        unpack8(make_uint4(wv[i][0], wv[i][1], wv[i][2], wv[i][3]), w);
    };
    auto measure = [&]() {
        sum = top = 0.0f;
#pragma unroll
        for (int i = 0; i < C; i++) {
            float w[8];
            weight(i, w);
#pragma unroll
            for (int z = 0; z < 8; z++) {
                sum = fmaf(h[i][z], h[i][z], sum);
                if (!FP8) top = fmaxf(top, fabsf(h[i][z] * w[z]));
            }
        }
        reduce_row<WAVE_ROW>(sum, top, lds);
    };
#pragma unroll
    for (int i = 0; i < C; i++) {
        unpack8(make_uint4(xv[i][0], xv[i][1], xv[i][2], xv[i][3]), h[i]);
        if (a.residual) {
            float r[8];
            unpack8(make_uint4(rv[i][0], rv[i][1], rv[i][2], rv[i][3]), r);
#pragma unroll
            for (int z = 0; z < 8; z++) h[i][z] += r[z];
        }
        const int u = tid + i * nt;
        if (a.sum && u < U)
            store16_nt(a.sum + at + 8 * u, bf16x8_of(h[i], 1.0f));
    }
    measure();
    float eps = a.eps;
    if (!(sum < kInf)) {
        top = 0.0f;
#pragma unroll
        for (int i = 0; i < C; i++)
#pragma unroll
            for (int z = 0; z < 8; z++) top = fmaxf(top, fabsf(h[i][z]));
        reduce_row<WAVE_ROW>(sum, top, lds);
        // the largest |h| to [2, 4); 0 for an infinite one, which makes NaN of it
        const float down = __uint_as_float((255u << 23) - (__float_as_uint(top) & 0x7F800000u));
#pragma unroll
        for (int i = 0; i < C; i++)
#pragma unroll
            for (int z = 0; z < 8; z++) h[i][z] *= down;
        eps = 0.0f;                            // at most 1, next to a mean past 2^111
        measure();
    }
    const bool finite = sum < kInf;
    // the reciprocal root of the unit, with one Newton step
    const float m = fmaf(sum, a.inv_h, eps);
    float r = __builtin_amdgcn_rsqf(m);
    r = fmaf(0.5f * r, fmaf(-m * r, r, 1.0f), r);
    r = finite ? r : __builtin_nanf("");
    constexpr float kTop = FP8 ? 448.0f : 127.0f;
    constexpr float kLeast = FP8 ? 0x1.cp-142f : 0x1.f8p-144f;   // the largest V with V / kTop == 0
#pragma unroll
    for (int i = 0; i < C; i++) {
        const int u = tid + i * nt;
        if (u >= U) break;
        float v[8], w[8];
        weight(i, w);
#pragma unroll
        for (int z = 0; z < 8; z++) v[z] = h[i][z] * w[z];
        if (a.y)
            store16_nt(a.y + at + 8 * u, bf16x8_of(v, r));
        if constexpr (FP8) {                   // 16 lanes hold a block of 128 channels
            top = 0.0f;
#pragma unroll
            for (int z = 0; z < 8; z++) top = fmaxf(top, fabsf(v[z]));
            top = group8_max(top);
            top = fmaxf(top, dpp_f32<kDppRowMirror>(top));
        }
        const float V = top * r;
        if (FP8 ? (u & 15) == 0 : u == 0)
            a.scales[FP8 ? t * (a.H / 128) + u / 16 : t] = V / kTop;
        // a value is multiplied by the factor's two parts (f from the reciprocal of the
        // unit, the rest from what it leaves), so the product is off by its own
        // rounding only
        float big = top;
        if (!(V > kLeast && top >= 0x1p-90f)) {
            // a scale that rounds to 0, or is NaN, has no codes; small values are first
            // brought to where the factor and its rest are normal
            const bool live = V > kLeast;
            big = live ? top * 0x1p100f : 1.0f;
#pragma unroll
            for (int z = 0; z < 8; z++) v[z] = live ? v[z] * 0x1p100f : 0.0f;
        }
        const float inv = __builtin_amdgcn_rcpf(big);
        const float f = kTop * inv, rest = fmaf(-f, big, kTop) * inv;
        float q[8];
#pragma unroll
        for (int z = 0; z < 8; z++) q[z] = fmaf(v[z], f, v[z] * rest);
        uint32_t code[2];
#pragma unroll
        for (int z = 0; z < 2; z++) {
            if constexpr (FP8) {               // |q| <= 448 (1 + 2^-23) rounds to at most 448
                int c = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * z], q[4 * z + 1], 0, false);
                code[z] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * z + 2], q[4 * z + 3], c, true);
            } else {
                code[z] = f32x4_to_int8(q[4 * z], q[4 * z + 1], q[4 * z + 2], q[4 * z + 3]);
            }
        }
        __builtin_nontemporal_store(u32x2{code[0], code[1]},
                                    reinterpret_cast<u32x2*>(a.out + at + 8 * u));
    }
}

}  // namespace

hipError_t launch_rmsnorm_quant(const NormArgs& a, hipStream_t stream, LaunchInfo* info, bool run) {
    const int U = a.H / 8;
    const bool wave_row = U <= 2 * kWave;
    const int C = wave_row ? (U <= kWave ? 1 : 2) : U <= 2048 ? 2 : U <= 4096 ? 4 : 8;
    const int threads = wave_row ? 256 : (U + C * kWave - 1) / (C * kWave) * kWave;
    const int64_t blocks = wave_row ? (a.T + 3) / 4 : a.T;
    if (info) *info = LaunchInfo{blocks, threads, 0, C, "rmsnorm_quant"};
    if (!run || blocks == 0) return hipSuccess;
    auto launch = [&](auto kernel) {
        kernel<<<dim3((unsigned)blocks), dim3(threads), 0, stream>>>(a);
    };
    auto pick = [&](auto fp8) {
        constexpr bool F = decltype(fp8)::value;
        if (wave_row) {
            if (C == 1) launch(k_rmsnorm_quant<F, 1, true>);
            else launch(k_rmsnorm_quant<F, 2, true>);
        } else {
            switch (C) {
                case 2: launch(k_rmsnorm_quant<F, 2, false>); break;
                case 4: launch(k_rmsnorm_quant<F, 4, false>); break;
                default: launch(k_rmsnorm_quant<F, 8, false>);
            }
        }
    };
    if (a.fp8) pick(std::true_type{});
    else pick(std::false_type{});
    return hipGetLastError();
}

}  // namespace moe
