// Grouped bf16 GEMM over the dispatch's bf16 segments, with bias, activation,
// gating and residual in the epilogue.
//
// Expert e owns rows [off[e], off[e+1]) of a. With z = a w[e]^T + bias[e] in
// fp32 over the whole inner dimension:
//
//   plain  y = act(z) + residual                          (N columns)
//   gated  y = act(z[:, :N/2]) * z[:, N/2:] + residual    (N/2 columns)
//
// and one rounding to bf16.
//
// Work split: segments are cut into tiles of kBM rows; a workgroup finds its
// tile by a scan over the segment lengths (no list kernel, no workspace) and
// computes one tile of 256 weight rows with 8 waves. In the gated form a
// wave's weight rows are half gate, half up of the same output columns, so
// the product is formed lane by lane. Each 64-wide k-block of both operands
// goes from memory straight into LDS (buffer_load ... lds) into a ring of
// stages; one barrier per k-block.
#include "activation.h"
#include "launch.h"
#include "moe_device.h"

#include <type_traits>

namespace moe {

namespace {

constexpr int kBN = 256;             // weight rows per tile
constexpr int kBK = 64;              // inner-dimension block: 128-byte rows in LDS
constexpr int kThreads = 512;
constexpr int kOutOfRange = 0x7FFFFF00;   // byte offset past every descriptor's end

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int chunk_key(int row) { return (row & 7) ^ ((row >> 3) & 1); }

template <int n>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(n >= 0 && n < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (n & 15) | ((n >> 4) << 14));
}

__device__ __forceinline__ void lds_barrier() { asm volatile("s_barrier" ::: "memory"); }

// Row tile `t` of the segments (counted over all experts in order) and the
// number of tiles. Segment bounds are clamped to the row capacity. Every
// thread of the workgroup takes part.
struct Tile {
    int row0, rows, e;
};

template <int BM>
__device__ __forceinline__ int find_tile(const int32_t* __restrict__ off, int E, int max_rows,
                                         int n_nt, int64_t item_of, Tile& out, int& nt_out) {
    __shared__ int s_wave[kThreads / kWave];
    __shared__ int s_tile[4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = tid >> 6;
    int r0[2], r1[2], n[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int e = 2 * tid + i;
        r0[i] = r1[i] = n[i] = 0;
        if (e < E) {
            r0[i] = min(max(off[e], 0), max_rows);
            r1[i] = min(max(off[e + 1], 0), max_rows);
            n[i] = r1[i] > r0[i] ? (r1[i] - r0[i] + BM - 1) / BM : 0;
        }
    }
    int incl = n[0] + n[1];
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int v = __shfl_up(incl, d, kWave);
        if (lane >= d) incl += v;
    }
    if (lane == 63) s_wave[wave] = incl;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / kWave; w++) {
        const int v = s_wave[w];
        before += w < wave ? v : 0;
        total += v;
    }
    const int64_t live = (int64_t)total * n_nt;
    if (item_of >= live) return 0;
    const int tile = (int)(item_of / n_nt);
    nt_out = (int)(item_of - (int64_t)tile * n_nt);
    int base = before + incl - n[0] - n[1];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        if (tile >= base && tile < base + n[i]) {
            s_tile[0] = r0[i] + (tile - base) * BM;
            s_tile[1] = min(BM, r1[i] - s_tile[0]);
            s_tile[2] = 2 * tid + i;
        }
        base += n[i];
    }
    __syncthreads();
    out.row0 = __builtin_amdgcn_readfirstlane(s_tile[0]);
    out.rows = __builtin_amdgcn_readfirstlane(s_tile[1]);
    out.e = __builtin_amdgcn_readfirstlane(s_tile[2]);
    return 1;
}

template <int BM>
struct Shape {
    static constexpr int kWavesM = BM / 64;
    static constexpr int kWavesN = 8 / kWavesM;
    static constexpr int kWaveCols = kBN / kWavesN;
    static constexpr int kJ = kWaveCols / 16;            // 16-column fragments per wave
    static constexpr int kStages = BM == 128 ? 3 : 2;
    static constexpr int kAChunks = BM / 64;             // 1 KB chunks per wave and stage
    static constexpr int kOps = kAChunks + 4;            // DMA loads per wave and stage
    static constexpr int kLds = kStages * (BM + kBN) * kBK * 2;
};

template <int BM, int ACT, bool GATED>
__global__ __launch_bounds__(kThreads, 1) void k_grouped_gemm_bf16(GemmBf16Args g) {
    using SH = Shape<BM>;
    constexpr int kStages = SH::kStages;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[SH::kLds];
    const int K = g.K;
    const int n_out = GATED ? g.N / 2 : g.N;             // output columns
    constexpr int kOutCols = GATED ? kBN / 2 : kBN;      // output columns per tile
    const int n_nt = (n_out + kOutCols - 1) / kOutCols;
    Tile td;
    int nt;
    if (!find_tile<BM>(g.off, g.E, (int)g.max_rows, n_nt, blockIdx.x, td, nt)) return;
    const int rows = td.rows;
    const int o0 = nt * kOutCols;
    const int KB = (K + kBK - 1) / kBK;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / SH::kWavesN, wn = wave % SH::kWavesN;

    // Rows past the tile's end, weight rows past N, and (by kOutOfRange)
    // columns past K read as zero.
    const auto ra = range_rsrc(g.a + (int64_t)td.row0 * K, rows * K * 2);
    const int cols = min(kOutCols, n_out - o0);
    // this wave's weight chunks: LDS rows 32 wave .. 32 wave + 31. LDS row r is
    // column (r / kWaveCols, r % kWaveCols) of the wave grid; in the gated
    // form the first half of each wave's columns are gate rows, the second up.
    constexpr int kHalf = SH::kWaveCols / 2;
    const int lrow = wave * 32;
    const int q = lrow % SH::kWaveCols;
    const bool up = GATED && q >= kHalf;
    const int col0 = GATED ? (lrow / SH::kWaveCols) * kHalf + q % kHalf : lrow;
    const auto rw = range_rsrc(
        g.w + ((int64_t)td.e * g.N + (up ? n_out : 0) + o0) * K, cols * K * 2);

    int a_goff[SH::kAChunks], w_goff[4];
#pragma unroll
    for (int i = 0; i < SH::kAChunks; i++) {
        const int p = (wave * SH::kAChunks + i) * 64 + lane, r = p >> 3;
        a_goff[i] = r * K * 2 + (((p & 7) ^ chunk_key(r)) << 4);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int p = (wave * 4 + i) * 64 + lane, r = p >> 3;
        w_goff[i] = (col0 + i * 8 + (lane >> 3)) * K * 2 + (((p & 7) ^ chunk_key(r)) << 4);
    }
    uint8_t* const sA = smem;
    uint8_t* const sW = smem + kStages * BM * 128;
    auto issue = [&](int st, int b) {
        const bool tail = (b + 1) * kBK > K;
#pragma unroll
        for (int i = 0; i < SH::kAChunks; i++) {
            int off = a_goff[i] + b * 128;
            const int r = (wave * SH::kAChunks + i) * 8 + (lane >> 3);
            if (tail && ((lane & 7) ^ chunk_key(r)) * 8 + b * kBK >= K) off = kOutOfRange;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                ra,
                (__attribute__((address_space(3))) void*)(sA + st * BM * 128 +
                                                          (wave * SH::kAChunks + i) * 1024),
                16, off, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            int off = w_goff[i] + b * 128;
            const int r = (wave * 4 + i) * 8 + (lane >> 3);
            if (tail && ((lane & 7) ^ chunk_key(r)) * 8 + b * kBK >= K) off = kOutOfRange;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rw,
                (__attribute__((address_space(3))) void*)(sW + st * kBN * 128 +
                                                          (wave * 4 + i) * 1024),
                16, off, 0, 0, 0);
        }
    };

    f32x4 acc[4][SH::kJ];
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < SH::kJ; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto frag = [&](const uint8_t* s, int row, int chunk) {
        return *reinterpret_cast<const bf16x8*>(s + row * 128 + ((chunk ^ chunk_key(row)) << 4));
    };
    constexpr int kAhead = kStages - 1;
#pragma unroll
    for (int s = 0; s < kAhead; s++) issue(s, min(s, KB - 1));
    int st = 0;
    for (int b = 0; b < KB; b++) {
        wait_vmcnt<SH::kOps*(kAhead - 1)>();
        lds_barrier();
        const int nst = st + kAhead >= kStages ? st + kAhead - kStages : st + kAhead;
        issue(nst, min(b + kAhead, KB - 1));
        const uint8_t* A = sA + st * BM * 128;
        const uint8_t* W = sW + st * kBN * 128;
#pragma unroll
        for (int kk = 0; kk < 2; kk++) {
            bf16x8 xf[4];
#pragma unroll
            for (int i = 0; i < 4; i++)
                xf[i] = frag(A, wm * 64 + i * 16 + (lane & 15), kk * 4 + (lane >> 4));
#pragma unroll
            for (int j = 0; j < SH::kJ; j++) {
                const bf16x8 wf =
                    frag(W, wn * SH::kWaveCols + j * 16 + (lane & 15), kk * 4 + (lane >> 4));
#pragma unroll
                for (int i = 0; i < 4; i++)
                    acc[i][j] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[i], acc[i][j], 0, 0, 0);
            }
        }
        st = st + 1 == kStages ? 0 : st + 1;
    }
    wait_vmcnt<0>();   // no LDS DMA may still be writing when the LDS is released

    // Lane: row 16i + lane%16, four consecutive columns 16j + 4 (lane/16) .. +3
    constexpr int kJOut = GATED ? SH::kJ / 2 : SH::kJ;
    const int c_wave = wn * (GATED ? kHalf : SH::kWaveCols) + 4 * (lane >> 4);
    const uint16_t* bias = g.bias ? g.bias + (int64_t)td.e * g.N : nullptr;
#pragma unroll
    for (int j = 0; j < kJOut; j++) {
        const int c = c_wave + j * 16;
        if (c >= cols) continue;
        float b0[4] = {0.f, 0.f, 0.f, 0.f}, b1[4] = {0.f, 0.f, 0.f, 0.f};
        if (bias) {
            const uint2 v = *reinterpret_cast<const uint2*>(bias + o0 + c);
            b0[0] = bf16_lo(v.x); b0[1] = bf16_hi(v.x); b0[2] = bf16_lo(v.y); b0[3] = bf16_hi(v.y);
            if constexpr (GATED) {
                const uint2 u = *reinterpret_cast<const uint2*>(bias + n_out + o0 + c);
                b1[0] = bf16_lo(u.x); b1[1] = bf16_hi(u.x);
                b1[2] = bf16_lo(u.y); b1[3] = bf16_hi(u.y);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int r = wm * 64 + i * 16 + (lane & 15);
            if (r >= rows) continue;
            float v[4];
#pragma unroll
            for (int x = 0; x < 4; x++) {
                v[x] = activate<ACT>(acc[i][j][x] + b0[x]);
                if constexpr (GATED) v[x] *= acc[i][j + kJOut][x] + b1[x];
            }
            const int64_t at = (int64_t)(td.row0 + r) * n_out + o0 + c;
            if (g.residual) {
                const uint2 u = *reinterpret_cast<const uint2*>(g.residual + at);
                v[0] += bf16_lo(u.x); v[1] += bf16_hi(u.x);
                v[2] += bf16_lo(u.y); v[3] += bf16_hi(u.y);
            }
            *reinterpret_cast<uint2*>(g.y + at) =
                make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]));
        }
    }
}

template <int BM, int ACT, bool GATED>
hipError_t run_shape(const GemmBf16Args& g, int64_t grid, hipStream_t stream) {
    k_grouped_gemm_bf16<BM, ACT, GATED><<<dim3((unsigned)grid), dim3(kThreads), 0, stream>>>(g);
    return hipGetLastError();
}

template <int BM, bool GATED>
hipError_t run_act(const GemmBf16Args& g, int64_t grid, hipStream_t stream) {
    switch (g.act) {
        case kActRelu: return run_shape<BM, kActRelu, GATED>(g, grid, stream);
        case kActSilu: return run_shape<BM, kActSilu, GATED>(g, grid, stream);
        case kActGelu: return run_shape<BM, kActGelu, GATED>(g, grid, stream);
        default: return run_shape<BM, kActNone, GATED>(g, grid, stream);
    }
}

}  // namespace

hipError_t launch_grouped_gemm_bf16(const GemmBf16Args& g, hipStream_t stream, LaunchInfo* info,
                                    bool run) {
    constexpr int BM = 128;
    const int n_out = g.gated ? g.N / 2 : g.N;
    const int out_cols = g.gated ? kBN / 2 : kBN;
    const int64_t max_tiles = (g.max_rows + BM - 1) / BM + g.E;
    const int64_t grid = max_tiles * ((n_out + out_cols - 1) / out_cols);
    if (info) *info = LaunchInfo{grid, kThreads, (size_t)Shape<BM>::kLds, BM, "grouped_gemm_bf16"};
    if (!run) return hipSuccess;
    return g.gated ? run_act<BM, true>(g, grid, stream)
                   : run_act<BM, false>(g, grid, stream);
}

}  // namespace moe
