// Scored router gate: sigmoid or softmax scores, a balance bias that enters
// the choice only, a choice limited to the best expert groups, top-k, and
// weights from the unbiased scores.
//
//   s[e]   = fp32(sigmoid(l[e]))  or  fp32(exp(l[e] - m) / sum exp(l - m))
//   key[e] = fp32(s[e] + bias[e]); a masked expert (logit or key -inf or NaN)
//            is never chosen
//   group score = fp32 sum of the group's group_top best live keys
//   chosen = the k best keys of the topk_group best groups
//   w[j]   = s[chosen j] (/ sum of the chosen scores) * scale
//
// Scores are rounded to fp32 once, from fp64: two neighbours at the border of
// the choice are often a few fp32 units apart, so a score that is one unit
// off would choose another expert. After that rounding the choice is exact
// fp32 comparisons and additions, ties to the lower index.
#include "launch.h"
#include "moe_device.h"

namespace moe {

namespace {

constexpr int kScoredThreads = 256;
constexpr int kScoredWaves = kScoredThreads / kWave;

__device__ __forceinline__ float load_logit(const void* p, bool bf16, int64_t i) {
    if (bf16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
    return static_cast<const float*>(p)[i];
}

struct DAdd {
    __device__ double operator()(double a, double b) const { return a + b; }
};

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
    return v;
}

// Order key of a selection value; 0 for one that can never be chosen.
__device__ __forceinline__ uint32_t choice_key(float v) {
    return v > -INFINITY ? order_key(v) : 0u;
}

}  // namespace

// One wave per token, experts lane, lane + 64, ... (any E, k, group count).
// LDS per wave: scores [E], keys [E] (reused by the group stage), chosen
// experts [k], group keys [n_group].
template <int NV>
__global__ __launch_bounds__(kScoredThreads) void k_route_scored(ScoredArgs a) {
    extern __shared__ uint32_t s_mem[];
    const int lane = threadIdx.x & (kWave - 1);
    const int wid = threadIdx.x / kWave;
    const int64_t t = (int64_t)blockIdx.x * kScoredWaves + wid;
    const bool live = t < a.T;
    const int E = a.E, k = a.k, ks = a.k + a.n_shared, G = a.n_group;
    uint32_t* mem = s_mem + (size_t)wid * (2 * E + k + G);
    float* s_score = reinterpret_cast<float*>(mem);
    uint32_t* s_key = mem + E;
    int32_t* s_sel = reinterpret_cast<int32_t*>(mem + 2 * E);
    uint32_t* s_group = mem + 2 * E + k;

    float l[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int e = lane + kWave * i;
        l[i] = (live && e < E) ? load_logit(a.logits, a.bf16, t * a.ld + e) : -INFINITY;
        if (!(l[i] > -INFINITY)) l[i] = -INFINITY;             // NaN: masked
    }
    float s[NV];
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < NV; i++) s[i] = (float)(1.0 / (1.0 + exp(-(double)l[i])));
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            l[i] = fminf(l[i], 3.402823466e38f);               // +inf: the largest finite value
            m = fmaxf(m, l[i]);
        }
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, kWave));
        double p[NV], sum = 0.0;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            p[i] = l[i] > -INFINITY ? exp((double)l[i] - (double)m) : 0.0;
            sum += p[i];
        }
        sum = wave_sum_f64(sum);
#pragma unroll
        for (int i = 0; i < NV; i++) s[i] = sum > 0.0 ? (float)(p[i] / sum) : 0.0f;
    }
    uint32_t c[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int e = lane + kWave * i;
        c[i] = 0u;
        if (e < E) {
            if (l[i] > -INFINITY) c[i] = choice_key(a.bias ? s[i] + a.bias[e] : s[i]);
            s_score[e] = s[i];
            s_key[e] = c[i];
        }
    }
    if (a.topk_group < G) {
        const int per = E / G;
        __syncthreads();
        for (int g = lane; g < G; g += kWave) {
            uint32_t k1 = 0u, k2 = 0u;
            for (int i = 0; i < per; i++) {
                const uint32_t v = s_key[g * per + i];
                k2 = v > k1 ? k1 : (v > k2 ? v : k2);
                k1 = v > k1 ? v : k1;
            }
            // the sum may be -inf only for keys near the lowest value: still live
            const float sc = (a.group_top == 2 && k2) ? key_value(k1) + key_value(k2) : key_value(k1);
            s_group[g] = k1 ? order_key(sc) : 0u;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int e = lane + kWave * i;
            if (e < E && c[i]) {
                const int g = e / per;
                const uint32_t mine = s_group[g];
                int rank = 0;
                for (int h = 0; h < G; h++) {
                    const uint32_t v = s_group[h];
                    rank += (v > mine || (v == mine && h < g)) ? 1 : 0;
                }
                if (rank >= a.topk_group) c[i] = 0u;
            }
        }
    }
    // k rounds: the wave's best key, ties to the lowest expert
    for (int r = 0; r < k; r++) {
        uint32_t best = c[0];
#pragma unroll
        for (int i = 1; i < NV; i++) best = best > c[i] ? best : c[i];
        const uint32_t m = group_reduce<kWave>(best, UMax());
        uint32_t e_min = 0xFFFFFFFFu;
#pragma unroll
        for (int i = NV - 1; i >= 0; i--)
            if (c[i] == m) e_min = (uint32_t)(lane + kWave * i);
        const uint32_t we = group_reduce<kWave>(e_min, UMin());
#pragma unroll
        for (int i = 0; i < NV; i++)
            if ((uint32_t)(lane + kWave * i) == we) c[i] = 0u;
        if (lane == 0) s_sel[r] = m ? (int32_t)we : -1;
    }
    __syncthreads();
    float part = 0.0f;
    for (int j = lane; j < k; j += kWave) {
        const int e = s_sel[j];
        part += e >= 0 ? s_score[e] : 0.0f;
    }
    const float total = __uint_as_float(group_reduce<kWave>(__float_as_uint(part), FAdd()));
    if (!live) return;
    for (int j = lane; j < k; j += kWave) {
        const int e = s_sel[j];
        float w = e >= 0 ? s_score[e] : 0.0f;
        if (a.renorm) w = total > 0.0f ? w / total : 0.0f;
        a.topk_idx[t * ks + j] = e;
        a.topk_w[t * ks + j] = w * a.scale;
    }
    for (int sh = lane; sh < a.n_shared; sh += kWave) {
        a.topk_idx[t * ks + k + sh] = E + sh;
        a.topk_w[t * ks + k + sh] = a.shared_w;
    }
}

hipError_t launch_route_scored(const ScoredArgs& a, hipStream_t stream, LaunchInfo* info,
                               bool run) {
    const int nv = (a.E + kWave - 1) / kWave;
    const int64_t blocks = (a.T + kScoredWaves - 1) / kScoredWaves;
    const size_t lds = (size_t)kScoredWaves * (2 * a.E + a.k + a.n_group) * 4;
    if (info) *info = LaunchInfo{blocks, kScoredThreads, lds, nv, "route_scored"};
    if (!run || blocks == 0) return hipSuccess;
    const dim3 grid((unsigned)blocks), block(kScoredThreads);
    if (nv <= 1) k_route_scored<1><<<grid, block, lds, stream>>>(a);
    else if (nv <= 2) k_route_scored<2><<<grid, block, lds, stream>>>(a);
    else if (nv <= 4) k_route_scored<4><<<grid, block, lds, stream>>>(a);
    else if (nv <= 8) k_route_scored<8><<<grid, block, lds, stream>>>(a);
    else k_route_scored<16><<<grid, block, lds, stream>>>(a);
    return hipGetLastError();
}

}  // namespace moe
