// Dispatch of rows that are already quantised, small batches: counting, the scan
// into offsets and the copy of codes and scales in one launch.
//
// Every workgroup reads the whole routing table (at most kDirectPairs slots) and
// counts it in LDS: one 32-bit counter an expert, the slots of all tokens in its
// lower half and those of the tokens before the workgroup's own in its upper half,
// by one atomic a slot. The lower halves, padded and scanned over the experts, are
// the segment offsets; offset plus upper half is the row of the workgroup's first
// slot of that expert, and each of its slots adds the number of those before it, so
// the order is the tokens'. The codes are on their way meanwhile. The table is small
// and comes from L2: no workgroup waits for another, and nothing is kept in a
// workspace.
//
// Against the counting, scanning and copying kernels, us: 1 token of 7168 bytes to 8
// of 256 experts 8.3 -> 4.8, 128 tokens 9.9 -> 5.7 (one launch instead of two); 2777
// tokens of 1408 bytes to 6 of 60, 16-row segments 19.6 -> 12.2, 4096 tokens of 1024
// to 8 of 256 21.2 -> 14.9 (instead of three). What is left is counting (in every
// workgroup, about 4 us at 16 thousand slots) next to the copy. Slots of one expert
// are counted one after the other, so the routing matters; see the rule below.
#include "launch.h"
#include "moe_device.h"

namespace moe {

namespace {

constexpr int kRowSlots = kMaxExperts;     // slots of a workgroup's tokens, at most
constexpr int kBatch = 4;                  // 16-byte loads of the table in flight

// Four slots of the table, which is aligned to one.
struct __attribute__((packed, aligned(4))) Quad {
    int e[4];
};

struct DirectPlan {
    int tokens;                            // of a workgroup
    int blocks, pad_parts, pad_per_expert, pad_rows;   // pad rows of an expert go in parts
};

template <int kThreads>
__global__ __launch_bounds__(kThreads) void k_dispatch_direct(DispatchArgs a, DirectPlan plan) {
    constexpr int kWaves = kThreads / kWave, kPerThread = kMaxExperts / kThreads;
    __shared__ uint32_t s_run[kMaxExperts];        // counters, then each expert's first row here
    __shared__ int s_cnt[kMaxExperts], s_off[kMaxExperts + 1], s_row[kRowSlots], s_wave[kWaves];
    __shared__ __attribute__((aligned(16))) int s_id[kRowSlots];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int E = a.E, k = a.k, T = (int)a.T;
    const int row_bytes = 2 * a.H, U = row_bytes / 16, CW = (U + kWave - 1) / kWave;
    const int t0 = min(T, (int)blockIdx.x * plan.tokens), nt = min(plan.tokens, T - t0);
    const uint8_t* const x = static_cast<const uint8_t*>(a.x);
    uint8_t* const out = static_cast<uint8_t*>(a.out);
    // item i of the workgroup: piece i % CW (64 lanes of 16 bytes) of token t0 + i / CW
    auto load = [&](int i) {
        const int64_t t = t0 + i / CW;
        return load16_nt(range_rsrc(x + t * row_bytes, row_bytes), 16 * ((i % CW) * kWave + lane));
    };
    const float first_scale = nt > 0 && a.scales == 1 ? a.x_scales[t0] : 0.0f;
    uint4 piece = make_uint4(0u, 0u, 0u, 0u);
    if (wave < nt * CW) piece = load(wave);

    for (int e = tid; e < E; e += kThreads) s_run[e] = 0;
    for (int p = tid; p < nt * k; p += kThreads) s_id[p] = a.topk_idx[t0 * k + p];
    __syncthreads();
    const int pairs = T * k, own = t0 * k, quads = pairs / 4;
    auto count = [&](int p, int e) {
        if ((unsigned)e < (unsigned)E) atomicAdd(&s_run[e], p < own ? 0x10001u : 1u);
    };
    for (int q0 = tid; q0 < quads; q0 += kBatch * kThreads) {
        Quad v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; i++) {
            const int q = q0 + i * kThreads;
            v[i] = Quad{{-1, -1, -1, -1}};
            if (q < quads) v[i] = reinterpret_cast<const Quad*>(a.topk_idx)[q];
        }
#pragma unroll
        for (int i = 0; i < kBatch; i++)
#pragma unroll
            for (int c = 0; c < 4; c++) count(4 * (q0 + i * kThreads) + c, v[i].e[c]);
    }
    if (tid < pairs - 4 * quads) count(4 * quads + tid, a.topk_idx[4 * quads + tid]);
    __syncthreads();
    int cnt[kPerThread], padded[kPerThread], sum = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; i++) {
        const int e = kPerThread * tid + i;
        cnt[i] = e < E ? (int)(s_run[e] & 0xFFFFu) : 0;
        padded[i] = (cnt[i] + a.row_align - 1) / a.row_align * a.row_align;
        sum += padded[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int v = __shfl_up(incl, d, kWave);
        if (lane >= d) incl += v;
    }
    if (lane == kWave - 1) s_wave[wave] = incl;
    __syncthreads();
    int at = incl - sum;
#pragma unroll
    for (int w = 0; w < kWaves; w++) at += w < wave ? s_wave[w] : 0;
#pragma unroll
    for (int i = 0; i < kPerThread; i++) {
        const int e = kPerThread * tid + i;
        if (e < E) {
            s_off[e] = at;
            s_cnt[e] = cnt[i];
            s_run[e] = at + (s_run[e] >> 16);
            if (blockIdx.x == 0) {
                a.expert_counts[e] = cnt[i];
                a.expert_offsets[e] = at;
            }
            if (e == E - 1) {
                s_off[E] = at + padded[i];
                if (blockIdx.x == 0) a.expert_offsets[E] = at + padded[i];
            }
        }
        at += padded[i];
    }
    __syncthreads();
    if (blockIdx.x == 0 && a.group_offsets != nullptr)
        for (int g = tid; g <= a.groups; g += kThreads)
            a.group_offsets[g] = s_off[g * (E / a.groups)];

    for (int p = tid; p < nt * k; p += kThreads) {
        const int e = s_id[p];
        int r = -1;
        if ((unsigned)e < (unsigned)E) {
            // the earlier slots of this workgroup's tokens with the same expert
            int rank = 0;
            for (int q = 0; q < p; q += 4) {
                const int4 v = *reinterpret_cast<const int4*>(s_id + q);
                rank += (v.x == e) + (v.y == e && q + 1 < p) + (v.z == e && q + 2 < p) +
                        (v.w == e && q + 3 < p);
            }
            r = (int)s_run[e] + rank;
            if (r < 0 || r >= a.max_rows) r = -1;            // never write outside
        }
        s_row[p] = r;
        a.dst_row[own + p] = r;
        if (r >= 0) {
            a.row_src[r] = own + p;
            if (a.scales == 1) a.out_scales[r] = nt == 1 ? first_scale : a.x_scales[t0 + p / k];
        }
    }
    __syncthreads();
    for (int i = wave; i < nt * CW; i += kWaves) {
        const int t = i / CW, u = (i % CW) * kWave + lane;
        if (i != wave) piece = load(i);
        for (int j = 0; j < k; j++) {
            const int r = __builtin_amdgcn_readfirstlane(s_row[t * k + j]);
            if (r >= 0 && u < U)
                store16_nt(out + (int64_t)r * row_bytes + 16 * (int64_t)u, piece);
        }
        if (a.scales > 1 && i % CW == 0) {
            for (int c = lane; c < a.scales; c += kWave) {
                const float s = a.x_scales[(int64_t)(t0 + t) * a.scales + c];
                for (int j = 0; j < k; j++) {
                    const int r = s_row[t * k + j];
                    if (r >= 0) a.out_scales[(int64_t)r * a.scales + c] = s;
                }
            }
        }
    }
    for (int pb = blockIdx.x; pb < plan.pad_parts; pb += plan.blocks) {
        const int e = pb / plan.pad_per_expert, part = pb % plan.pad_per_expert;
        const int first = s_off[e] + s_cnt[e] + part * plan.pad_rows;
        const int rows = min(s_off[e + 1] - first, plan.pad_rows);
        for (int i = tid; i < rows * U; i += kThreads)
            *reinterpret_cast<uint4*>(out + (int64_t)first * row_bytes + 16 * (int64_t)i) =
                make_uint4(0u, 0u, 0u, 0u);
        for (int i = tid; i < rows * a.scales; i += kThreads)
            a.out_scales[(int64_t)first * a.scales + i] = 0.0f;
        for (int i = tid; i < rows; i += kThreads) a.row_src[first + i] = -1;
    }
}

}  // namespace

// Up to kDirectPairs slots (the counters' halves hold 65535), and no more than 2048 an
// expert on average, or 4096 with one choice a token, where the kernels have more tokens
// to pass over. us here / by the counting, scanning and copying kernels, rows of 512 bytes,
// popularity of a spread of 0.5:
//   slots        4096         8192        16384        32768
//   1 of 1     12.1/13.2    19.8/15.3    34.9/21.2    66.8/33.4
//   1 of 4      9.4/13.3    14.5/15.7    24.9/21.7    45.8/34.1
//   1 of 8      7.9/13.4    11.0/15.7    17.9/21.7    31.9/34.5
//   2 of 2     10.7/9.3     17.0/13.9    29.3/16.7    54.5/23.0
//   2 of 8      7.7/9.5     10.5/14.3    16.3/17.1    28.2/23.7
//   4 of 8      7.6/9.7      9.9/10.2    14.5/15.5    24.1/19.2
//   8 of 8      6.6/10.2     9.4/11.1    13.1/11.9    20.8/17.8
//   8 of 16     6.3/10.1     8.7/11.0    11.8/11.9    17.9/17.7
//   8 of 32     6.0/10.1     8.3/11.2    11.0/12.0    15.9/17.8
// The host does not know how the slots are spread: 32768 x 1 of 8 take 24.5 (evenly), 51
// (popularity of a spread of 3) or 67 (all to one) against 34; 4096 x 8 of 256, rows of
// 1024, 14.6 or 19.8 against 19.4. With 48 to 65 thousand slots what is gained shrinks
// (8191 x 8 of 256, rows of 1024: 26.0/29.4; of 32: 30.1/28.9).
bool dispatch_direct_applies(int64_t T, int E, int k) {
    return T * k <= kDirectPairs && T * k <= (k == 1 ? 4096 : 2048) * (int64_t)E;
}

hipError_t launch_dispatch_direct(const DispatchArgs& a, hipStream_t stream, LaunchInfo* info,
                                  bool run) {
    DirectPlan plan;
    // One workgroup a token while all of them run at once, then more tokens each, since
    // every workgroup counts the whole table. Up to 768 tokens four workgroups of 512
    // threads a CU, then two of 1024, which count half as often. us, tokens x choices of
    // experts, bytes a row:             4 of 512  2 of 1024
    //     128 x 8 of 256, 7168             5.8       6.0
    //     700 x 8 of 128, 2048             7.6       7.7
    //    1024 x 8 of 256, 1024             8.8       8.1
    //    2777 x 6 of 60, 1408, 16-row     14.8      12.2
    //    4096 x 8 of 256, 1024            17.5      14.9
    //   32768 x 1 of 8, 512               35.4      25.2
    const bool wide = a.T > 768;
    const int most = wide ? 512 : 1024;
    // Slots of a workgroup: k of one token, at most kMaxExperts; or, past 768 tokens,
    // where k <= 32768 / 769, fewer than k (T / 512 + 1) <= 64 + 42.
    const int64_t tokens = (a.T + most - 1) / most;
    plan.tokens = tokens < 1 ? 1 : (int)tokens;
    plan.pad_per_expert = a.T > 0 && a.row_align > 1 ? (a.row_align - 1 < 4 ? a.row_align - 1 : 4) : 0;
    plan.pad_parts = a.E * plan.pad_per_expert;
    plan.pad_rows = plan.pad_parts ? (a.row_align + plan.pad_per_expert - 2) / plan.pad_per_expert : 0;
    const int64_t token_blocks = (a.T + plan.tokens - 1) / plan.tokens;
    const int64_t least = plan.pad_parts < most ? plan.pad_parts : most;
    plan.blocks = (int)(token_blocks > least ? token_blocks : least);
    if (plan.blocks < 1) plan.blocks = 1;              // no tokens: the tables
    const int threads = wide ? 1024 : 512;
    if (info) *info = LaunchInfo{plan.blocks, threads, 0, plan.tokens, "count+scan+scatter"};
    if (!run) return hipSuccess;
    const dim3 grid((unsigned)plan.blocks), block(threads);
    if (wide) k_dispatch_direct<1024><<<grid, block, 0, stream>>>(a, plan);
    else k_dispatch_direct<512><<<grid, block, 0, stream>>>(a, plan);
    return hipGetLastError();
}

}  // namespace moe
