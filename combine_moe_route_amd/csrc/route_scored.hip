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
//
// Two kernels. k_route_chunks cuts a row into chunks of four experts and takes k
// up to 64, rows at most 2^20 elements apart and at most 256 chunks, where each
// group's count is filled up to a power of two; the choice is k rounds of a
// maximum over the lanes of a token, or sorting networks. k_route_rounds takes
// the rest: k above 64, rows further apart, and wide groups whose filled counts
// pass 256 (five groups of 129 to 204 experts: 5 x 64).
#include "launch.h"
#include "moe_device.h"
#include "topk_sort.h"

namespace moe {

namespace {

constexpr int kScoredThreads = 256;
constexpr int kScoredWaves = kScoredThreads / kWave;

__device__ __forceinline__ float load_logit(const void* p, bool bf16, int64_t i) {
    if (bf16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
    return static_cast<const float*>(p)[i];
}

struct FMax {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
};

// exp(y) in fp64 for |y| <= 150: y = n ln 2 + r with |r| <= ln 2 / 2 (Cody and
// Waite's reduction, ln 2 in two parts), the Taylor series of exp(r) to
// r^12 / 12! (the next term is below 2^-52), times 2^n.
// A score rounded to fp32 from it differs from the right rounding only where
// the exact value lies within about 2^-51 of a midpoint between two floats,
// once in 2^25 values.
__device__ __forceinline__ double exp64(double y) {
    const double n = rint(y * 1.4426950408889634);
    double r = fma(n, -0.69314718055994530942, y);       // ln 2 as a double,
    r = fma(n, -2.3190468138462996e-17, r);              // and what it lacks
    double p = 2.08767569878680989792e-09;               // 1 / 12!
    p = fma(p, r, 2.50521083854417187751e-08);
    p = fma(p, r, 2.75573192239858906526e-07);
    p = fma(p, r, 2.75573192239858906526e-06);
    p = fma(p, r, 2.48015873015873015873e-05);
    p = fma(p, r, 1.98412698412698412698e-04);
    p = fma(p, r, 1.38888888888888888889e-03);
    p = fma(p, r, 8.33333333333333333333e-03);
    p = fma(p, r, 4.16666666666666666667e-02);
    p = fma(p, r, 1.66666666666666666667e-01);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return ldexp(p, (int)n);
}

// 1 / d for d in [1, 2^220]: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double recip64(double d) {
    double q = __builtin_amdgcn_rcp(d);
    q = fma(fma(-d, q, 1.0), q, q);
    return fma(fma(-d, q, 1.0), q, q);
}

// Beyond +-150 the score is 0 or 1 in fp32 already.
__device__ __forceinline__ float sigmoid32(float l) {
    return (float)recip64(1.0 + exp64(-(double)__builtin_amdgcn_fmed3f(l, -150.0f, 150.0f)));
}

// exp(l - m) for l <= m; below exp(-150) nothing reaches an fp32 score
__device__ __forceinline__ double exp_diff(float l, float m) {
    return exp64(fmax((double)l - (double)m, -150.0));
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
    return v;
}

// Candidate of an order key and a position below 1024, as in topk_sort.h.
__device__ __forceinline__ double key_pack(uint32_t key, int pos) {
    return __hiloint2double((int)__builtin_amdgcn_alignbit(0x400u, key, 12),
                            (int)((key << 20) | (uint32_t)(1023 - pos)));
}

// Order key of a selection value; 0 for one that can never be chosen.
__device__ __forceinline__ uint32_t choice_key(float v) {
    return v > -INFINITY ? order_key(v) : 0u;
}

}  // namespace

// One wave per token, experts lane, lane + 64, ... (any E, k, group count). With
// groups, lane g scans group g serially.
// LDS per wave: scores [E], keys [E] (reused by the group stage), chosen
// experts [k], group keys [n_group].
template <int NV>
__global__ __launch_bounds__(kScoredThreads) void k_route_rounds(ScoredArgs a) {
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
        for (int i = 0; i < NV; i++) s[i] = sigmoid32(l[i]);
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
            p[i] = l[i] > -INFINITY ? exp_diff(l[i], m) : 0.0;
            sum += p[i];
        }
        sum = wave_sum_f64(sum);
        const double inv = sum > 0.0 ? recip64(sum) : 0.0;
#pragma unroll
        for (int i = 0; i < NV; i++) s[i] = (float)(p[i] * inv);
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

// ------------------------------------------------------------------ chunks

namespace {

constexpr int kPast = 0x7FFFFF00;    // byte offset past every descriptor's end

// How k_route_chunks lays a row out; lanes == 0: the shape is not for it.
struct ChunkPlan {
    int lanes;   // per token
    int rows;    // chunks per lane
    int sorted;  // sorting networks instead of rounds (rows == 4, k <= kList)
    int cg_lg;   // slots per group: 1 << cg_lg, the last ones empty
    int wide;    // chunks are whole and aligned for one load each
};

constexpr int kList = 8;             // candidates the sorting networks keep

// The list of the 2 D lanes a butterfly step joins; across rows of 16 lanes both
// rows' lists come from one swap.
template <int D>
__device__ __forceinline__ void join_lists(double (&list)[kList]) {
    if constexpr (D < 16) {
        merge_with_partner<D, kList>(list);
    } else {
        double other[kList];
#pragma unroll
        for (int q = 0; q < kList; q++) {
            const uint32_t hi = (uint32_t)__double2hiint(list[q]);
            const uint32_t lo = (uint32_t)__double2loint(list[q]);
            const auto h = D == 16 ? __builtin_amdgcn_permlane16_swap(hi, hi, false, false)
                                   : __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
            const auto l = D == 16 ? __builtin_amdgcn_permlane16_swap(lo, lo, false, false)
                                   : __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
            list[q] = __hiloint2double((int)h[0], (int)l[0]);
            other[q] = __hiloint2double((int)h[1], (int)l[1]);
        }
        merge_top<kList>(list, other);
    }
}

// The two largest of a1 >= a2 and the partner's pair b1 >= b2.
__device__ __forceinline__ void two_best(float& a1, float& a2, float b1, float b2) {
    const float lo = fminf(a1, b1);
    a1 = fmaxf(a1, b1);
    a2 = fmaxf(lo, fmaxf(a2, b2));
}

// The value of the lane across from this one in a butterfly of 2 D lanes; for
// D >= 4 any lane of the other half (they hold the same by then).
template <int D>
__device__ __forceinline__ float across(float v) {
    if constexpr (D == 1) return dpp_f32<kDppQuadXor1>(v);
    else if constexpr (D == 2) return dpp_f32<kDppQuadXor2>(v);
    else if constexpr (D == 4) return dpp_f32<kDppRowHalfMirror>(v);
    else if constexpr (D == 8) return dpp_f32<kDppRowMirror>(v);
    else return __shfl_xor(v, D, kWave);
}

}  // namespace

// S lanes per token, R chunks of four experts per lane: slot g + S i is row i of
// lane g. A group of experts has 1 << cg_lg slots (without groups the whole row
// is one), so its slots are neighbouring lanes, or whole rows, and its two best
// keys are a butterfly over them. Slots ascend with the experts, so a tie goes
// to the lower position 4 slot + x.
//
// The k best, SORTED: a lane sorts its 16 candidates, packed with their positions
// into doubles as in topk_sort.h, down to a list of 8, and the lists of the
// token's lanes are merged by a butterfly. Otherwise in k rounds: the best key
// of a lane, the maximum over the token's lanes (DPP, permlane swaps), and the
// position of its holder, by ballot and readlane where a wave holds one token
// and the maximum is unique, else a minimum over the lanes. Lane r keeps the
// winner of round r.
//
// Large batches are bound by instructions: 16384 tokens, 256 experts in 8 groups,
// k 8, sigmoid with bias take 103 vector instructions a logit and lane, about 26 of
// them the fp64 score; at four cycles each they fill 79 % of the cycles (counters).
// 5003 tokens of 160 experts in groups are bound by latency: 59 %, 2.4 waves per
// SIMD, which wait half of their time. The first case takes 14.5 us (1.2 TB/s; the
// first kernel, one token per wave with the device library's exp and a serial group
// scan, took 29.9 us), one token 4.1 us (7.3 us). Tried: sorting with 8 lanes
// per token and keys waiting in LDS, 19.2 us and 13.0 us; every lane then works
// through 32 experts in series.
template <int S, int R, bool SORTED, bool SIGMOID, bool GROUPED>
__global__ __launch_bounds__(kScoredThreads) void k_route_chunks(ScoredArgs a, ChunkPlan p) {
    __shared__ float4 s_score[R][kScoredThreads];        // [row][lane of every token]
    __shared__ uint32_t s_group[GROUPED ? kScoredThreads * R : 1];
    constexpr int kTokens = kScoredThreads / S;
    const int tid = threadIdx.x, g = tid & (S - 1), tl = tid / S;
    const int64_t t0 = (int64_t)blockIdx.x * kTokens;
    const int64_t t = t0 + tl;
    const bool live = t < a.T;
    const int E = a.E, k = a.k, ks = a.k + a.n_shared;
    const int per = GROUPED ? E / a.n_group : E;
    const int cg_mask = (1 << p.cg_lg) - 1;
    const int size = a.bf16 ? 2 : 4;

    // this block's rows of logits, bounded by the last one's end
    const int64_t left = a.T - t0;
    const int64_t block_rows = left < kTokens ? left : kTokens;
    const auto rs = range_rsrc(static_cast<const char*>(a.logits) + t0 * a.ld * size,
                               (int)(((block_rows - 1) * a.ld + E) * size));
    const int row_off = live ? (int)(tl * a.ld) * size : kPast;
    int e0[R], n[R];                                     // first expert, experts held
#pragma unroll
    for (int i = 0; i < R; i++) {
        const int slot = g + S * i;
        const int group = GROUPED ? slot >> p.cg_lg : 0;
        const int in = GROUPED ? slot & cg_mask : slot;
        e0[i] = group * per + 4 * in;
        n[i] = !GROUPED || group < a.n_group ? per - 4 * in : 0;
    }
    float l[R][4];
    if (p.wide && a.bf16) {
        uint32_t u[R][2];
#pragma unroll
        for (int i = 0; i < R; i++) {
            const auto h = __builtin_amdgcn_raw_buffer_load_b64(
                rs, live && n[i] > 0 ? row_off + e0[i] * 2 : kPast, 0, 0);
            u[i][0] = h[0];
            u[i][1] = h[1];
        }
#pragma unroll
        for (int i = 0; i < R; i++) {
            l[i][0] = bf16_lo(u[i][0]);
            l[i][1] = bf16_hi(u[i][0]);
            l[i][2] = bf16_lo(u[i][1]);
            l[i][3] = bf16_hi(u[i][1]);
        }
    } else if (p.wide) {
        u32x4 u[R];
#pragma unroll
        for (int i = 0; i < R; i++)
            u[i] = __builtin_amdgcn_raw_buffer_load_b128(
                rs, live && n[i] > 0 ? row_off + e0[i] * 4 : kPast, 0, 0);
#pragma unroll
        for (int i = 0; i < R; i++)
#pragma unroll
            for (int x = 0; x < 4; x++) l[i][x] = __uint_as_float(u[i][x]);
    } else if (a.bf16) {
#pragma unroll
        for (int i = 0; i < R; i++)
#pragma unroll
            for (int x = 0; x < 4; x++)
                l[i][x] = bf16_lo((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
                    rs, live && x < n[i] ? row_off + (e0[i] + x) * 2 : kPast, 0, 0));
    } else {
#pragma unroll
        for (int i = 0; i < R; i++)
#pragma unroll
            for (int x = 0; x < 4; x++)
                l[i][x] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                    rs, live && x < n[i] ? row_off + (e0[i] + x) * 4 : kPast, 0, 0));
    }
    const auto rb = range_rsrc(a.bias, a.bias ? E * 4 : 0);   // no bias: zeros
    float b[R][4];
#pragma unroll
    for (int i = 0; i < R; i++)
#pragma unroll
        for (int x = 0; x < 4; x++)
            b[i][x] = __uint_as_float(
                __builtin_amdgcn_raw_buffer_load_b32(rb, (e0[i] + x) * 4, 0, 0));

    // scores; masked logits (-inf, NaN) and empty places as -inf
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < R; i++)
#pragma unroll
        for (int x = 0; x < 4; x++) {
            // +inf: the largest finite value in the softmax
            if (!SIGMOID) l[i][x] = l[i][x] > 3.402823466e38f ? 3.402823466e38f : l[i][x];
            l[i][x] = (x < n[i]) & (l[i][x] > -INFINITY) ? l[i][x] : -INFINITY;
            m = fmaxf(m, l[i][x]);
        }
    float s[R][4];
    if constexpr (SIGMOID) {
#pragma unroll
        for (int i = 0; i < R; i++)
#pragma unroll
            for (int x = 0; x < 4; x++) s[i][x] = sigmoid32(l[i][x]);
    } else {
        m = __uint_as_float(group_reduce<S>(__float_as_uint(m), FMax()));
        double pr[R][4], sum = 0.0;
#pragma unroll
        for (int i = 0; i < R; i++)
#pragma unroll
            for (int x = 0; x < 4; x++) {
                pr[i][x] = exp_diff(l[i][x], m);         // a masked one: exp(-150), nothing
                sum += pr[i][x];
            }
#pragma unroll
        for (int d = 1; d < S; d <<= 1) sum += __shfl_xor(sum, d, kWave);
        const double inv = recip64(sum);
#pragma unroll
        for (int i = 0; i < R; i++)
#pragma unroll
            for (int x = 0; x < 4; x++) s[i][x] = (float)(pr[i][x] * inv);
    }
    uint32_t c[R][4];                                    // choice keys, 0: never chosen
    float key[R][4];
#pragma unroll
    for (int i = 0; i < R; i++) {
        s_score[i][tid] = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
#pragma unroll
        for (int x = 0; x < 4; x++) {
            key[i][x] = s[i][x] + b[i][x];
            key[i][x] = (l[i][x] > -INFINITY) & (key[i][x] > -INFINITY) ? key[i][x] : -INFINITY;
            c[i][x] = key[i][x] > -INFINITY ? order_key(key[i][x]) : 0u;
        }
    }

    if constexpr (GROUPED) {
        float t1[R], t2[R];
#pragma unroll
        for (int i = 0; i < R; i++) {
            t1[i] = fmaxf(key[i][0], key[i][1]);
            t2[i] = fminf(key[i][0], key[i][1]);
            two_best(t1[i], t2[i], fmaxf(key[i][2], key[i][3]), fminf(key[i][2], key[i][3]));
            if (p.cg_lg > 0) two_best(t1[i], t2[i], across<1>(t1[i]), across<1>(t2[i]));
            if (p.cg_lg > 1) two_best(t1[i], t2[i], across<2>(t1[i]), across<2>(t2[i]));
            if (p.cg_lg > 2) two_best(t1[i], t2[i], across<4>(t1[i]), across<4>(t2[i]));
            if (S > 8 && p.cg_lg > 3) two_best(t1[i], t2[i], across<8>(t1[i]), across<8>(t2[i]));
            if (S > 16 && p.cg_lg > 4) two_best(t1[i], t2[i], across<16>(t1[i]), across<16>(t2[i]));
            if (S > 32 && p.cg_lg > 5) two_best(t1[i], t2[i], across<32>(t1[i]), across<32>(t2[i]));
        }
        // a group of more slots than lanes is two rows (there are at most four)
        if (R > 2 && 1 << p.cg_lg > S) {
#pragma unroll
            for (int i = 0; i + 1 < R; i += 2) {
                two_best(t1[i], t2[i], t1[i + 1], t2[i + 1]);
                t1[i + 1] = t1[i];
                t2[i + 1] = t2[i];
            }
        }
        uint32_t gk[R];
        uint32_t* const mine = s_group + tl * (S * R);
#pragma unroll
        for (int i = 0; i < R; i++) {
            const int slot = g + S * i;
            gk[i] = t1[i] > -INFINITY
                ? order_key(a.group_top == 2 && t2[i] > -INFINITY ? t1[i] + t2[i] : t1[i]) : 0u;
            if ((slot & cg_mask) == 0) mine[slot >> p.cg_lg] = gk[i];
        }
        __syncthreads();
        int before[R];                                   // groups that rank before this one
#pragma unroll
        for (int i = 0; i < R; i++) before[i] = 0;
#pragma unroll 4
        for (int o = 0; o < a.n_group; o++) {
            const uint32_t v = mine[o];
#pragma unroll
            for (int i = 0; i < R; i++)
                before[i] += (v > gk[i]) | ((v == gk[i]) & (o < ((g + S * i) >> p.cg_lg))) ? 1 : 0;
        }
#pragma unroll
        for (int i = 0; i < R; i++)
#pragma unroll
            for (int x = 0; x < 4; x++) c[i][x] = before[i] < a.topk_group ? c[i][x] : 0u;
    }

    uint32_t sel_key = 0u, sel_pos = 0u;
    if constexpr (SORTED) {
        static_assert(R == 4, "sixteen candidates a lane");
        double list[kList], more[kList];
#pragma unroll
        for (int q = 0; q < kList; q++) {
            const int i = q / 4, x = q % 4;
            const int at = 4 * (g + S * i) + x, below = 4 * (g + S * (i + 2)) + x;
            list[q] = c[i][x] ? key_pack(c[i][x], at) : kCandNone;
            more[q] = c[i + 2][x] ? key_pack(c[i + 2][x], below) : kCandNone;
        }
        sort_desc<kList>(list);
        sort_desc<kList>(more);
        merge_top<kList>(list, more);
        join_lists<1>(list);
        join_lists<2>(list);
        join_lists<4>(list);
        if constexpr (S > 8) join_lists<8>(list);
        if constexpr (S > 16) join_lists<16>(list);
        if constexpr (S > 32) join_lists<32>(list);
#pragma unroll
        for (int r = 0; r < kList; r++) {
            sel_key = g == r ? cand_key(list[r]) : sel_key;
            sel_pos = g == r ? (uint32_t)cand_expert(list[r]) : sel_pos;
        }
    } else {
        for (int r = 0; r < k; r++) {
            uint32_t best = 0u;
#pragma unroll
            for (int i = 0; i < R; i++)
#pragma unroll
                for (int x = 0; x < 4; x++) best = best > c[i][x] ? best : c[i][x];
            const uint32_t top = group_reduce<S>(best, UMax());
            uint32_t pos = 0xFFFFFFFFu;                      // this lane's lowest holder
#pragma unroll
            for (int i = R - 1; i >= 0; i--)
#pragma unroll
                for (int x = 3; x >= 0; x--) pos = c[i][x] == top ? 4u * (g + S * i) + x : pos;
            if constexpr (S == kWave) {
                const uint64_t mask = __ballot(best == top);
                if (__popcll(mask) == 1)
                    pos = (uint32_t)__builtin_amdgcn_readlane((int)pos, (int)__builtin_ctzll(mask));
                else
                    pos = group_reduce<S>(pos, UMin());
            } else {
                pos = group_reduce<S>(pos, UMin());
            }
#pragma unroll
            for (int i = 0; i < R; i++)
#pragma unroll
                for (int x = 0; x < 4; x++) c[i][x] = pos == 4u * (g + S * i) + x ? 0u : c[i][x];
            sel_key = g == r ? top : sel_key;
            sel_pos = g == r ? pos : sel_pos;
        }
    }

    // weights: lane r has slot r
    __syncthreads();
    const bool mine = g < k && sel_key != 0u;
    const int slot = (int)(sel_pos >> 2);
    const float* const row = reinterpret_cast<const float*>(
        &s_score[mine ? slot / S : 0][tl * S + (mine ? slot & (S - 1) : 0)]);
    float w = mine ? row[sel_pos & 3] : 0.0f;
    const float total = __uint_as_float(group_reduce<S>(__float_as_uint(w), FAdd()));
    if (!live) return;
    if (g < k) {
        const int e = (GROUPED ? (slot >> p.cg_lg) * per + 4 * (slot & cg_mask) : 4 * slot) +
                      (int)(sel_pos & 3);
        if (a.renorm) w = total > 0.0f ? w / total : 0.0f;
        a.topk_idx[t * ks + g] = mine ? e : -1;
        a.topk_w[t * ks + g] = w * a.scale;
    }
    for (int sh = g; sh < a.n_shared; sh += S) {
        a.topk_idx[t * ks + k + sh] = E + sh;
        a.topk_w[t * ks + k + sh] = a.shared_w;
    }
}

namespace {

ChunkPlan chunk_plan(const ScoredArgs& a) {
    ChunkPlan p{0, 1, 0, 0, 0};
    const bool grouped = a.topk_group < a.n_group;
    const int per = grouped ? a.E / a.n_group : a.E;
    while (4 << p.cg_lg < per) p.cg_lg++;
    const int slots = grouped ? a.n_group << p.cg_lg : (per + 3) / 4;
    // a block's rows have to fit a buffer descriptor
    if (slots > 4 * kWave || a.k > kWave || a.ld > (1 << 20)) return p;
    // One chunk per lane is quickest for one token; where many tokens share the
    // chip, fewer lanes with more chunks save instructions. Half the lanes: 16384
    // tokens of 256 experts 19.0 -> 16.8 us (sigmoid, 8 groups), 17.3 -> 14.4 us
    // (softmax, no groups). Four chunks a lane through the sorting networks: 14.5
    // and 11.2 us; 2048 tokens of 384 experts 6.9 -> 5.2 us; but 6.4 -> 7.2 us for
    // 4096 tokens of 160 experts in groups (too few waves to hide the chains),
    // and 4.9 -> 6.7 us for 16384 tokens of 64 experts (mostly empty places).
    int lanes = 8;
    while (lanes < kWave && (lanes < slots || lanes < a.k)) lanes <<= 1;
    if (a.T >= 2048 && lanes > 8 && lanes / 2 >= a.k && slots <= lanes * 2) lanes >>= 1;
    if (slots > 16 && a.k <= kList) {
        int four = 8;
        while (four * 4 < slots) four <<= 1;
        p.sorted = a.T * four >= (grouped ? 1 << 17 : 1 << 16);
        if (p.sorted) {
            lanes = four;
            p.rows = 4;
        }
    }
    while (p.rows * lanes < slots) p.rows <<= 1;
    p.lanes = lanes;
    const uintptr_t base = reinterpret_cast<uintptr_t>(a.logits);
    p.wide = per % 4 == 0 && (!a.bf16 || (a.ld % 2 == 0 && base % 4 == 0));
    return p;
}

template <int S, int R, bool SORTED = false>
void launch_chunks(const ScoredArgs& a, const ChunkPlan& p, int64_t blocks, hipStream_t stream) {
    const dim3 grid((unsigned)blocks), block(kScoredThreads);
    const bool grouped = a.topk_group < a.n_group;
    if (a.sigmoid && grouped) k_route_chunks<S, R, SORTED, true, true><<<grid, block, 0, stream>>>(a, p);
    else if (a.sigmoid) k_route_chunks<S, R, SORTED, true, false><<<grid, block, 0, stream>>>(a, p);
    else if (grouped) k_route_chunks<S, R, SORTED, false, true><<<grid, block, 0, stream>>>(a, p);
    else k_route_chunks<S, R, SORTED, false, false><<<grid, block, 0, stream>>>(a, p);
}

}  // namespace

hipError_t launch_route_scored(const ScoredArgs& a, hipStream_t stream, LaunchInfo* info,
                               bool run) {
    const ChunkPlan p = chunk_plan(a);
    if (p.lanes) {
        const int64_t per_block = kScoredThreads / p.lanes;
        const int64_t blocks = (a.T + per_block - 1) / per_block;
        if (info) *info = LaunchInfo{blocks, kScoredThreads, 0, p.lanes, "route_chunks"};
        if (!run || blocks == 0) return hipSuccess;
        if (p.sorted) {
            switch (p.lanes) {
                case 8: launch_chunks<8, 4, true>(a, p, blocks, stream); break;
                case 16: launch_chunks<16, 4, true>(a, p, blocks, stream); break;
                case 32: launch_chunks<32, 4, true>(a, p, blocks, stream); break;
                default: launch_chunks<64, 4, true>(a, p, blocks, stream);
            }
            return hipGetLastError();
        }
        switch (p.lanes * 8 + p.rows) {
            case 8 * 8 + 1: launch_chunks<8, 1>(a, p, blocks, stream); break;
            case 16 * 8 + 1: launch_chunks<16, 1>(a, p, blocks, stream); break;
            case 32 * 8 + 1: launch_chunks<32, 1>(a, p, blocks, stream); break;
            case 8 * 8 + 2: launch_chunks<8, 2>(a, p, blocks, stream); break;
            case 16 * 8 + 2: launch_chunks<16, 2>(a, p, blocks, stream); break;
            case 32 * 8 + 2: launch_chunks<32, 2>(a, p, blocks, stream); break;
            case 32 * 8 + 4: launch_chunks<32, 4>(a, p, blocks, stream); break;
            case 64 * 8 + 1: launch_chunks<64, 1>(a, p, blocks, stream); break;
            case 64 * 8 + 2: launch_chunks<64, 2>(a, p, blocks, stream); break;
            default: launch_chunks<64, 4>(a, p, blocks, stream);
        }
        return hipGetLastError();
    }
    const int nv = (a.E + kWave - 1) / kWave;
    const int64_t blocks = (a.T + kScoredWaves - 1) / kScoredWaves;
    const size_t lds = (size_t)kScoredWaves * (2 * a.E + a.k + a.n_group) * 4;
    if (info) *info = LaunchInfo{blocks, kScoredThreads, lds, nv, "route_rounds"};
    if (!run || blocks == 0) return hipSuccess;
    const dim3 grid((unsigned)blocks), block(kScoredThreads);
    if (nv <= 1) k_route_rounds<1><<<grid, block, lds, stream>>>(a);
    else if (nv <= 2) k_route_rounds<2><<<grid, block, lds, stream>>>(a);
    else if (nv <= 4) k_route_rounds<4><<<grid, block, lds, stream>>>(a);
    else if (nv <= 8) k_route_rounds<8><<<grid, block, lds, stream>>>(a);
    else k_route_rounds<16><<<grid, block, lds, stream>>>(a);
    return hipGetLastError();
}

}  // namespace moe
