// Tiles of the grouped GEMMs whose operands are plain rows (bf16, int8): finding
// a workgroup's tile, the pipelined product, the skinny product for few rows, and
// the epilogue. The products differ in the matrix instruction only: a fragment is
// 16 bytes of a row a lane in both, so everything that moves data counts in
// 2-byte units (K bf16 values, or pairs of int8 values).
#pragma once

#include "activation.h"
#include "launch.h"
#include "moe_device.h"

#include <type_traits>

namespace moe {

namespace {

constexpr int kBK = 64;              // inner-dimension block in 2-byte units: 128-byte rows in LDS
constexpr int kXcds = 8;             // workgroup b runs on XCD b mod 8
constexpr int kBand = 4;             // row tiles that take the same weights one after the other
// A byte offset past every descriptor (256 rows of 2^20 bf16: 2^29 bytes), which
// stays below 2^31 with any row offset within a tile added.
constexpr int kOutOfRange = 0x60000000;

// The products: a lane's fragment of 16 bytes, its 16 sums, the instruction, and
// whether the sums are scaled by row and by column.
struct Bf16 {
    typedef __bf16 Frag __attribute__((ext_vector_type(8)));
    typedef float Acc __attribute__((ext_vector_type(16)));
    typedef float Acc4 __attribute__((ext_vector_type(4)));
    static constexpr bool kScaled = false;
    static constexpr const char* kName = "grouped_gemm_bf16";
    static constexpr const char* kStreamedName = "streamed_grouped_gemm_bf16";
    static __device__ __forceinline__ Acc mma(Frag w, Frag x, Acc c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, x, c, 0, 0, 0);
    }
};
struct Int8 {
    typedef int Frag __attribute__((ext_vector_type(4)));
    typedef int Acc __attribute__((ext_vector_type(16)));
    typedef int Acc4 __attribute__((ext_vector_type(4)));
    static constexpr bool kScaled = true;
    static constexpr const char* kName = "grouped_gemm_int8";
    static constexpr const char* kStreamedName = "streamed_grouped_gemm_int8";
    static __device__ __forceinline__ Acc mma(Frag w, Frag x, Acc c) {
        return __builtin_amdgcn_mfma_i32_32x32x32_i8(w, x, c, 0, 0, 0);
    }
};

// LDS layout of a staged k-block: 128-byte rows of eight 16-byte chunks, chunk
// c of row r at physical chunk c ^ key(r). A fragment read has lanes 32 q + l
// at (row l, chunk 2 s + q); the hardware serves it 16 lanes at a time, rows
// {0..3, 12..15, 20..27} or {4..11, 16..19, 28..31} of one chunk. Two rows
// share 256 bytes (all banks), so the eight even rows of such a group, like
// the eight odd ones, need distinct chunks, which this key gives (counters: no
// conflict; a layout made for sixteen rows in sequence had one per access).
__device__ __forceinline__ int chunk_key(int row) { return row >> 1 & 7; }

template <int n>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(n >= 0 && n < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (n & 15) | ((n >> 4) << 14));
}

__device__ __forceinline__ void lds_barrier() { asm volatile("s_barrier" ::: "memory"); }

// f(integral_constant 0), ..., f(integral_constant N - 1)
template <int N, typename F>
__device__ __forceinline__ void unrolled(F f) {
    if constexpr (N > 0) {
        unrolled<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

// Rows row0 .. row0 + rows - 1 of expert e.
struct Tile {
    int row0, rows, e;
};

// This workgroup's row tile and column tile; false if it has none. Segment
// bounds are clamped to the row capacity; every thread takes part. Tiles are
// numbered expert by expert; within one, bands of kBand row tiles run through
// the column tiles together, column by column, so that the weights of a column
// tile are read by neighbours in time. The workgroups of one XCD (b mod kXcds)
// take a contiguous run of the numbers, so that this happens in one L2
// (7.95 -> 7.45 ms for 16384 tokens over 256 experts; bands of 3, 4 and 8: 7.52,
// 7.45 and 7.39 ms there, but 729, 713 and 737 us for one segment of 16384 rows).
template <int BM, int THREADS>
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ off, int E, int max_rows,
                                          int n_nt, int* scratch, Tile& out, int& nt_out) {
    constexpr int kPer = kMaxExperts / THREADS;          // experts per thread
    int* s_wave = scratch;                               // [THREADS / kWave]
    int* s_tile = scratch + THREADS / kWave;             // [4]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = tid >> 6;
    int r0[kPer], r1[kPer], n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int e = kPer * tid + i;
        r0[i] = r1[i] = n[i] = 0;
        if (e < E) {
            r0[i] = min(max(off[e], 0), max_rows);
            r1[i] = min(max(off[e + 1], 0), max_rows);
            n[i] = r1[i] > r0[i] ? (r1[i] - r0[i] - 1) / BM + 1 : 0;
        }
        sum += n[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int v = __shfl_up(incl, d, kWave);
        if (lane >= d) incl += v;
    }
    if (lane == 63) s_wave[wave] = incl;
    if (tid == 0) s_tile[0] = s_tile[1] = s_tile[2] = s_tile[3] = 0;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / kWave; w++) {
        const int v = s_wave[w];
        before += w < wave ? v : 0;
        total += v;
    }
    const int64_t live = (int64_t)total * n_nt;
    const int64_t chunk = (live + kXcds - 1) / kXcds;
    const int64_t local = blockIdx.x / kXcds;
    const int64_t item = (blockIdx.x % kXcds) * chunk + local;
    if (local >= chunk || item >= live) return false;
    int64_t base = (int64_t)(before + incl - sum) * n_nt;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        if (item >= base && item < base + (int64_t)n[i] * n_nt) {
            const int q = (int)(item - base);
            const int first = q / (kBand * n_nt) * kBand;
            const int band = min(kBand, n[i] - first), in = q - first * n_nt;
            const int t = first + in % band;
            s_tile[0] = r0[i] + t * BM;
            s_tile[1] = min(BM, r1[i] - s_tile[0]);
            s_tile[2] = kPer * tid + i;
            s_tile[3] = in / band;
        }
        base += (int64_t)n[i] * n_nt;
    }
    __syncthreads();
    out.row0 = __builtin_amdgcn_readfirstlane(s_tile[0]);
    out.rows = __builtin_amdgcn_readfirstlane(s_tile[1]);
    out.e = __builtin_amdgcn_readfirstlane(s_tile[2]);
    nt_out = __builtin_amdgcn_readfirstlane(s_tile[3]);
    // offsets that do not ascend can name no tile, or more than one
    out.rows = min(out.rows, max_rows - out.row0);
    __syncthreads();                                     // the scratch is free again
    return out.rows > 0;
}

// Eight bf16 values at p (16-byte aligned) to fp32.
__device__ __forceinline__ void load8(const uint16_t* p, float* f) {
    unpack8(*reinterpret_cast<const uint4*>(p), f);
}

// N fp32 values at p (16-byte aligned).
template <int N>
__device__ __forceinline__ void load_f32(const float* p, float* f) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + i);
        f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
    }
}

// A sum in fp32, with the scales of its row and column where the product has
// them: the whole number is rounded to fp32 once, then each scale multiplied in,
// the row's first (a product of the two scales alone could underflow).
template <typename P, typename T>
__device__ __forceinline__ float scaled(T sum, float row, float column) {
    if constexpr (P::kScaled) return (float)sum * row * column;
    else return sum;
}

// Scales, bias, activation, gate, residual and the rounding of one wave's tile of
// IF x JF fragments at (wm, wn). A lane holds, for fragment (i, j), row
// 32 i + lane % 32 and the 16 columns 32 j + 16 (lane / 32) .. +15 (the weight
// rows are staged in that order), so that residual and result move in 16-byte
// pieces.
template <typename P, int IF, int JF, int ACT, bool GATED>
__device__ __forceinline__ void epilogue(const GroupedGemmArgs& g, const Tile& td, int o0, int cols,
                                         int wm, int wn, const typename P::Acc (&acc)[IF][JF]) {
    constexpr int kJOut = GATED ? JF / 2 : JF;
    const int lane = threadIdx.x & 63;
    const int n_out = GATED ? g.N / 2 : g.N;
    const int c_lane = wn * kJOut * 32 + 16 * (lane >> 5);
    const int r_lane = wm * IF * 32 + (lane & 31);
    const uint16_t* bias = g.bias ? g.bias + (int64_t)td.e * g.N + o0 : nullptr;
    const int64_t at0 = (int64_t)(td.row0 + r_lane) * n_out + o0;
    const float* ws = P::kScaled ? g.w_scales + (int64_t)td.e * g.N + o0 : nullptr;
    float as[IF];
    if constexpr (P::kScaled)
#pragma unroll
        for (int i = 0; i < IF; i++)
            as[i] = r_lane + i * 32 < td.rows ? g.a_scales[td.row0 + r_lane + i * 32] : 0.0f;
    // residual pieces are loaded one 32-column group ahead of their use
    uint4 res[2][2][IF];
    auto load_res = [&](int j) {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int i = 0; i < IF; i++)
                if (c_lane + j * 32 + h * 8 < cols && r_lane + i * 32 < td.rows)
                    res[j & 1][h][i] = *reinterpret_cast<const uint4*>(
                        g.residual + at0 + (int64_t)i * 32 * n_out + c_lane + j * 32 + h * 8);
    };
    if (g.residual) load_res(0);
#pragma unroll
    for (int j = 0; j < kJOut; j++) {
        if (g.residual && j + 1 < kJOut) load_res(j + 1);
#pragma unroll
        for (int h = 0; h < 2; h++) {                    // N is a multiple of 8: whole pieces
            const int c = c_lane + j * 32 + h * 8;
            if (c >= cols) continue;
            float b0[8], b1[8], s0[8], s1[8];
#pragma unroll
            for (int z = 0; z < 8; z++) b0[z] = b1[z] = 0.0f;
            if (bias) {
                load8(bias + c, b0);
                if constexpr (GATED) load8(bias + n_out + c, b1);
            }
            if constexpr (P::kScaled) {
                load_f32<8>(ws + c, s0);
                if constexpr (GATED) load_f32<8>(ws + n_out + c, s1);
            }
#pragma unroll
            for (int i = 0; i < IF; i++) {
                if (r_lane + i * 32 >= td.rows) continue;
                float v[8];
#pragma unroll
                for (int z = 0; z < 8; z++) {
                    v[z] = activate<ACT>(scaled<P>(acc[i][j][8 * h + z], as[i], s0[z]) + b0[z]);
                    if constexpr (GATED)
                        v[z] *= scaled<P>(acc[i][j + kJOut][8 * h + z], as[i], s1[z]) + b1[z];
                }
                if (g.residual) {
                    float f[8];
                    unpack8(res[j & 1][h][i], f);
#pragma unroll
                    for (int z = 0; z < 8; z++) v[z] += f[z];
                }
                *reinterpret_cast<uint4*>(g.y + at0 + (int64_t)i * 32 * n_out + c) =
                    make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]),
                               cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
            }
        }
    }
}

// ------------------------------------------------------------------ many rows

// One tile of WM IF 32 rows and WN JF 32 weight rows with WM x WN waves of
// IF x JF fragments, over rings of SA LDS stages of activations and SW of weights
// (an array each, so that the compiler can tell the DMA into one from reads of
// another; else it drains all DMA before every read). A k-block is multiplied in
// two halves of 32; while a wave multiplies one half it reads the fragments of
// the next into its other register set, so no product waits for LDS. One barrier
// per k-block, between the halves: every wave has then read all of k-block b, so
// the activations of b + SA go into its stage during the second half, and the
// weights of b + SW into its stage during the first half of b + 1. Loads are
// spread over the products, so that no wave queues behind its own.
template <typename P, int SA, int SW, int WM, int WN, int IF, int JF, bool GATED>
__device__ __forceinline__ void tile_body(const GroupedGemmArgs& g, const Tile& td, int nt,
                                          uint8_t* const (&sA)[SA], uint8_t* const (&sW)[SW]) {
    static_assert(SA >= 2 && (SW == SA || SW == SA + 1), "stages");
    constexpr int U = SA == SW ? SA : SA * SW;           // steps until the stages repeat
    constexpr int kWaves = WM * WN, kBN = WN * JF * 32;
    constexpr int kAOps = WM * IF * 4 / kWaves;          // 1 KB DMA pieces (8 rows) per wave
    constexpr int kWOps = kBN / 8 / kWaves;
    const int K = g.K, KB = (K + kBK - 1) / kBK;
    const int n_out = GATED ? g.N / 2 : g.N;
    const int o0 = nt * (GATED ? kBN / 2 : kBN);
    const int cols = min(GATED ? kBN / 2 : kBN, n_out - o0);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    // Rows past the tile's end, weight rows past N, and (by kOutOfRange)
    // columns past K read as zero. LDS weight row r belongs to wave column
    // r / (32 JF); in the gated form the first half of a wave column's rows
    // are gate rows, the second half up rows of the same outputs (a wave
    // stages rows of one kind only).
    constexpr int kCols = JF * 32, kHalf = kCols / 2;
    static_assert(!GATED || kHalf % (kWOps * 8) == 0, "one kind of weight row per wave");
    // Within 32 rows, row 8 x + 4 h + z holds column 16 h + 4 x + z: a lane of
    // the product then has 16 consecutive columns.
    const int lrow = wave * kWOps * 8;                   // first weight row this wave stages
    static_assert(kWOps % 4 == 0, "a wave stages whole groups of 32 weight rows");
    const bool up = GATED && lrow % kCols >= kHalf;
    const int col0 = GATED ? lrow / kCols * kHalf + lrow % kHalf : lrow;
    const auto ra = range_rsrc(g.a + (int64_t)td.row0 * K, td.rows * K * 2);
    const auto rw = range_rsrc(g.w + ((int64_t)td.e * g.N + (up ? n_out : 0) + o0) * K,
                               cols * K * 2);
    // LDS 16-byte slot p of a stage is (row p / 8, physical chunk p % 8); the
    // keys repeat every 16 rows, so two offsets serve all pieces
    static_assert(kAOps % 2 == 0 && kWOps % 2 == 0, "a wave's pieces start at a multiple of 16 rows");
    int a_off[2], w_off[2], kc[2];                       // kc: this lane's first column
#pragma unroll
    for (int i = 0; i < 2; i++) {
        kc[i] = ((lane & 7) ^ chunk_key(i * 8 + (lane >> 3))) * 8;
        a_off[i] = (wave * kAOps * 8 + (lane >> 3)) * K * 2 + kc[i] * 2;
        w_off[i] = (col0 + 16 * (lane >> 5) + (lane >> 3 & 3)) * K * 2 + kc[i] * 2;
    }
    auto issue_a = [&](int st, int b) {
        int v[2];
#pragma unroll
        for (int i = 0; i < 2; i++)
            v[i] = (b + 1) * kBK > K && kc[i] + b * kBK >= K ? kOutOfRange : a_off[i] + b * kBK * 2;
#pragma unroll
        for (int i = 0; i < kAOps; i++)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                ra, (__attribute__((address_space(3))) void*)(sA[st] + (wave * kAOps + i) * 1024),
                16, v[i & 1] + i * 16 * K, 0, 0, 0);
    };
    auto issue_w = [&](int st, int b) {
        int v[2];
#pragma unroll
        for (int i = 0; i < 2; i++)
            v[i] = (b + 1) * kBK > K && kc[i] + b * kBK >= K ? kOutOfRange : w_off[i] + b * kBK * 2;
#pragma unroll
        for (int i = 0; i < kWOps; i++)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rw, (__attribute__((address_space(3))) void*)(sW[st] + (wave * kWOps + i) * 1024),
                16, v[i & 1] + (i / 4 * 32 + i % 4 * 4) * 2 * K, 0, 0, 0);
    };
    typename P::Acc acc[IF][JF];
#pragma unroll
    for (int i = 0; i < IF; i++)
#pragma unroll
        for (int j = 0; j < JF; j++)
#pragma unroll
            for (int x = 0; x < 16; x++) acc[i][j][x] = 0;
    // fragment: rows lane % 32 (+ 32 i), chunk 2 s + lane / 32 of step s; the
    // key depends on the row within 16 only
    using Frag = typename P::Frag;
    Frag xf[2][2][IF], wf[2][2][JF];                     // [half][step of 32 bytes]
    const int fr = (lane & 31) * 128;
    int fc[4];
#pragma unroll
    for (int s = 0; s < 4; s++) fc[s] = fr + ((2 * s + (lane >> 5)) ^ chunk_key(lane & 31)) * 16;
    auto read = [&](auto half, int st) {                 // st: step number mod U
        constexpr int H = decltype(half)::value;
#pragma unroll
        for (int s = 0; s < 2; s++) {
            const uint8_t* pa = sA[st % SA] + wm * IF * 4096 + fc[2 * H + s];
            const uint8_t* pw = sW[st % SW] + wn * JF * 4096 + fc[2 * H + s];
#pragma unroll
            for (int j = 0; j < JF; j++)
                wf[H][s][j] = *reinterpret_cast<const Frag*>(pw + j * 4096);
#pragma unroll
            for (int i = 0; i < IF; i++)
                xf[H][s][i] = *reinterpret_cast<const Frag*>(pa + i * 4096);
        }
    };
    auto mma = [&](auto half) {
        constexpr int H = decltype(half)::value;
#pragma unroll
        for (int s = 0; s < 2; s++)
#pragma unroll
            for (int i = 0; i < IF; i++)
#pragma unroll
                for (int j = 0; j < JF; j++)
                    acc[i][j] = P::mma(wf[H][s][j], xf[H][s][i], acc[i][j]);
    };
    using H0 = std::integral_constant<int, 0>;
    using H1 = std::integral_constant<int, 1>;
    constexpr int kReads = 2 * (IF + JF), kMfma = 2 * IF * JF;
    constexpr int kLeft = kAOps * (SA - 2) + kWOps * (SW - 2);
    // products, LDS reads and DMA loads of a half in even measure
    auto interleave = [&](auto loads) {
        constexpr int D = decltype(loads)::value;
        static_assert(D <= kReads, "at most one load per LDS read");
#pragma unroll
        for (int x = 0; x < kReads; x++) {
            if (x < kMfma)
                __builtin_amdgcn_sched_group_barrier(0x008, kMfma < kReads ? 1 : kMfma / kReads, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                  // LDS read
            if (x * D % kReads < D) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);   // load
        }
    };
    auto step = [&](auto stage, int b) {
        constexpr int ST = decltype(stage)::value;
        __builtin_amdgcn_sched_barrier(0);
        issue_w((ST + SW - 1) % SW, min(b + SW - 1, KB - 1));   // the stage of b - 1
        read(H1{}, ST);
        mma(H0{});
        interleave(std::integral_constant<int, kWOps>{});
        // this wave's pieces of k-block b + 1 have landed and its fragments of
        // b are in registers; after the barrier that holds for every wave
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0x0070 | (kLeft & 15) | ((kLeft >> 4) << 14));
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        issue_a(ST % SA, min(b + SA, KB - 1));
        read(H0{}, ST + 1);
        mma(H1{});
        interleave(std::integral_constant<int, kAOps>{});
    };
#pragma unroll
    for (int st = 0; st < SA; st++) {                    // in the order of use
        issue_a(st, min(st, KB - 1));
        if (st < SW - 1) issue_w(st, min(st, KB - 1));
    }
    wait_vmcnt<kAOps*(SA - 1) + kWOps*(SW - 2)>();
    lds_barrier();
    read(H0{}, 0);
    // a wave whose rows all lie past the tile's end only moves data
    auto over_k = [&](auto f) {
        int b = 0;
        for (; b + U <= KB; b += U) unrolled<U>([&](auto st) { f(st, b + decltype(st)::value); });
        unrolled<U - 1>([&](auto st) {
            if (b + decltype(st)::value < KB) f(st, b + decltype(st)::value);
        });
    };
    if (wm * IF * 32 < td.rows) {
        over_k(step);
    } else {
        over_k([&](auto stage, int b) {
            constexpr int ST = decltype(stage)::value;
            issue_w((ST + SW - 1) % SW, min(b + SW - 1, KB - 1));
            wait_vmcnt<kLeft>();
            lds_barrier();
            issue_a(ST % SA, min(b + SA, KB - 1));
        });
    }
    wait_vmcnt<0>();   // no LDS DMA may still be writing when the LDS is released
    switch (g.act) {
        case kActRelu: epilogue<P, IF, JF, kActRelu, GATED>(g, td, o0, cols, wm, wn, acc); break;
        case kActSilu: epilogue<P, IF, JF, kActSilu, GATED>(g, td, o0, cols, wm, wn, acc); break;
        case kActGelu: epilogue<P, IF, JF, kActGelu, GATED>(g, td, o0, cols, wm, wn, acc); break;
        default: epilogue<P, IF, JF, kActNone, GATED>(g, td, o0, cols, wm, wn, acc);
    }
}

// Tile shapes (rows x weight rows), waves, LDS stages of A and W:
//   Large   256 x 256, 4 waves of 128 x 128, 2 + 3, one workgroup per CU
//   Medium  128 x 256, 8 waves of 64 x 64, 3 + 3, one per CU
//   Small   128 x 128, 4 waves of 64 x 64, 2 + 3, two per CU
//   Skinny  32 x 64 (or x 32), see below, two per CU or more; STREAM loads the
//           weights with the non-temporal hint
struct Large {
    static constexpr int kBM = 256, kBN = 256, kThreads = 256, kLds = 163840;
};
struct Medium {
    static constexpr int kBM = 128, kBN = 256, kThreads = 512, kLds = 147456;
};
struct Small {
    static constexpr int kBM = 128, kBN = 128, kThreads = 256, kLds = 81920;
};
template <bool STREAM, int BN = 64>
struct Skinny {
    static constexpr int kBM = 32, kBN = BN, kThreads = 256, kLds = 1024 * BN;
    static constexpr bool kStream = STREAM;
};

template <typename P, typename SH, bool GATED>
__global__ __launch_bounds__(SH::kThreads, SH::kLds > 81920 ? 1 : 2) void k_grouped_gemm(
    GroupedGemmArgs g) {
    constexpr int kA = SH::kBM * kBK * 2, kW = SH::kBN * kBK * 2;
    __shared__ __attribute__((aligned(1024))) uint8_t a0[kA], a1[kA], w0[kW], w1[kW], w2[kW];
    const int n_out = GATED ? g.N / 2 : g.N;
    constexpr int kOutCols = GATED ? SH::kBN / 2 : SH::kBN;
    Tile td;
    int nt;
    if (!find_tile<SH::kBM, SH::kThreads>(g.off, g.E, (int)g.max_rows,
                                          (n_out + kOutCols - 1) / kOutCols,
                                          reinterpret_cast<int*>(a0), td, nt))
        return;
    uint8_t* const sW[3] = {w0, w1, w2};
    if constexpr (std::is_same_v<SH, Medium>) {
        __shared__ __attribute__((aligned(1024))) uint8_t a2[kA];
        uint8_t* const sA[3] = {a0, a1, a2};
        tile_body<P, 3, 3, 2, 4, 2, 2, GATED>(g, td, nt, sA, sW);
    } else {
        uint8_t* const sA[2] = {a0, a1};
        if constexpr (std::is_same_v<SH, Large>)
            tile_body<P, 2, 3, 2, 2, 4, 4, GATED>(g, td, nt, sA, sW);
        else
            tile_body<P, 2, 3, 2, 2, 2, 2, GATED>(g, td, nt, sA, sW);
    }
}

// ------------------------------------------------------------------ few rows

// Scales, bias, activation, gate, residual and rounding of four columns of a row.
template <typename P, int ACT, bool GATED>
__device__ __forceinline__ void skinny_store(const GroupedGemmArgs& g, const Tile& td, int o0,
                                             int cols, const typename P::Acc4& z0,
                                             const typename P::Acc4& z1) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n_out = GATED ? g.N / 2 : g.N;
    const int r = lane & 31;
    if (r >= td.rows) return;
    const uint16_t* bias = g.bias ? g.bias + (int64_t)td.e * g.N + o0 : nullptr;
    const float* ws = P::kScaled ? g.w_scales + (int64_t)td.e * g.N + o0 : nullptr;
    const float as = P::kScaled ? g.a_scales[td.row0 + r] : 0.0f;
#pragma unroll
    for (int j = 0; j < (GATED ? 1 : 2); j++) {
        const int c = 32 * j + 16 * (lane >> 5) + 4 * wave;
        if (c >= cols) continue;
        float b0[4] = {0.f, 0.f, 0.f, 0.f}, b1[4] = {0.f, 0.f, 0.f, 0.f};
        if (bias) {
            const uint2 v = *reinterpret_cast<const uint2*>(bias + c);
            b0[0] = bf16_lo(v.x); b0[1] = bf16_hi(v.x); b0[2] = bf16_lo(v.y); b0[3] = bf16_hi(v.y);
            if constexpr (GATED) {
                const uint2 u = *reinterpret_cast<const uint2*>(bias + n_out + c);
                b1[0] = bf16_lo(u.x); b1[1] = bf16_hi(u.x);
                b1[2] = bf16_lo(u.y); b1[3] = bf16_hi(u.y);
            }
        }
        float v[4], s0[4], s1[4];
        if constexpr (P::kScaled) {
            load_f32<4>(ws + c, s0);
            if constexpr (GATED) load_f32<4>(ws + n_out + c, s1);
        }
#pragma unroll
        for (int z = 0; z < 4; z++) {
            v[z] = activate<ACT>(scaled<P>(j ? z1[z] : z0[z], as, s0[z]) + b0[z]);
            if constexpr (GATED) v[z] *= scaled<P>(z1[z], as, s1[z]) + b1[z];
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

// One tile of 32 rows and 64 (or 32) weight rows; the inner dimension is split over
// the 4 waves (wave w takes k-blocks w, w + 4, ...), which read nothing of each
// other until their sums are joined at the end. A wave streams its weight
// k-blocks through two LDS stages of its own and holds the activations of the
// same k-blocks in registers (a fragment is 16 bytes a lane, straight from the
// row), so it meets no barrier and two workgroups fit a CU.
template <typename P, typename SH, bool GATED>
__global__ __launch_bounds__(SH::kThreads, 2) void k_grouped_gemm_skinny(GroupedGemmArgs g) {
    constexpr bool STREAM = SH::kStream;
    constexpr int kWaves = 4, JF = SH::kBN / 32;         // groups of 32 weight rows
    static_assert(JF == 2 || (JF == 1 && !GATED), "gate and up rows are a group each");
    constexpr int kStage = SH::kBN * kBK * 2;            // 8 KB of weights, or 4
    __shared__ __attribute__((aligned(1024))) uint8_t s0[kWaves * kStage], s1[kWaves * kStage];
    const int K = g.K, KB = (K + kBK - 1) / kBK;
    const int n_out = GATED ? g.N / 2 : g.N;
    constexpr int kOutCols = GATED ? 32 : SH::kBN;
    Tile td;
    int nt;
    if (!find_tile<32, SH::kThreads>(g.off, g.E, (int)g.max_rows,
                                         (n_out + kOutCols - 1) / kOutCols,
                                         reinterpret_cast<int*>(s0), td, nt))
        return;
    const int o0 = nt * kOutCols;
    const int cols = min(kOutCols, n_out - o0);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const auto ra = range_rsrc(g.a + (int64_t)td.row0 * K, td.rows * K * 2);
    // two groups of 32 weight rows: gate and up, or columns 0..31 and 32..63
    const uint16_t* const wp = g.w + ((int64_t)td.e * g.N + o0) * K;
    const __amdgpu_buffer_rsrc_t rw[2] = {
        range_rsrc(wp, min(32, cols) * K * 2),
        GATED ? range_rsrc(wp + (int64_t)n_out * K, cols * K * 2)
              : range_rsrc(wp + (int64_t)32 * K, max(0, cols - 32) * K * 2)};
    int w_off[2], kc[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        kc[i] = ((lane & 7) ^ chunk_key(i * 8 + (lane >> 3))) * 8;
        w_off[i] = (16 * (lane >> 5) + (lane >> 3 & 3)) * K * 2 + kc[i] * 2;
    }
    const int a_row = (lane & 31) * K * 2;
    u32x4 af[2][4];
    // this wave's k-blocks: wave + kWaves ((i + turn) mod n). Every tile starts at
    // another place, so that workgroups that run in step do not all read the
    // same columns of rows a power of two apart, which are the same memory
    // channels (one token through 2 of 8 experts, K 4096, N 16384: 46 us, without
    // this 67; K 7168 is not affected).
    const int n = (KB - wave + kWaves - 1) / kWaves;
    const int turn = n > 0 ? nt % n : 0;
    auto issue = [&](auto stage, int i) {
        constexpr int ST = decltype(stage)::value;
        int at = i + turn;
        at -= at >= n ? n : 0;
        const int k0 = i < n ? (wave + kWaves * at) * kBK : K;   // K: all zero
        uint8_t* s = (ST ? s1 : s0) + wave * kStage;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int c = k0 + (2 * q + (lane >> 5)) * 8;
            af[ST][q] = __builtin_amdgcn_raw_buffer_load_b128(
                ra, c < K ? a_row + c * 2 : kOutOfRange, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4 * JF; i++)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rw[i / 4], (__attribute__((address_space(3))) void*)(s + i * 1024), 16,
                k0 + kc[i & 1] < K ? w_off[i & 1] + i % 4 * 8 * K + k0 * 2 : kOutOfRange, 0, 0,
                STREAM ? kCachePolicyNT : 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    using Frag = typename P::Frag;
    using Acc4 = typename P::Acc4;
    typename P::Acc acc[JF];
#pragma unroll
    for (int j = 0; j < JF; j++)
#pragma unroll
        for (int x = 0; x < 16; x++) acc[j][x] = 0;
    const int fr = (lane & 31) * 128;
    auto step = [&](auto stage, int i) {
        constexpr int ST = decltype(stage)::value;
        wait_vmcnt<4 + 4 * JF>();                        // all but the k-block behind this one
        __builtin_amdgcn_sched_barrier(0);
        const uint8_t* s = (ST ? s1 : s0) + wave * kStage + fr;
        Frag wf[4][JF];
#pragma unroll
        for (int q = 0; q < 4; q++)
#pragma unroll
            for (int j = 0; j < JF; j++)
                wf[q][j] = *reinterpret_cast<const Frag*>(
                    s + j * 4096 + (((2 * q + (lane >> 5)) ^ chunk_key(lane & 31)) << 4));
#pragma unroll
        for (int q = 0; q < 4; q++)
#pragma unroll
            for (int j = 0; j < JF; j++)
                acc[j] = P::mma(wf[q][j], __builtin_bit_cast(Frag, af[ST][q]), acc[j]);
        issue(stage, i + 2);
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    if (n > 0) {
        issue(S0{}, 0);
        issue(S1{}, 1);
        for (int i = 0; i < n; i += 2) {
            step(S0{}, i);
            if (i + 1 < n) step(S1{}, i + 1);
        }
    }
    wait_vmcnt<0>();
    // join: wave w finishes columns 16 h + 4 w .. +3 of every row, from the
    // four waves' sums in order
    Acc4* const join = reinterpret_cast<Acc4*>(s0);      // [wave][j][x / 4][lane], 16 KB a group
    __syncthreads();
#pragma unroll
    for (int j = 0; j < JF; j++)
#pragma unroll
        for (int x = 0; x < 4; x++)
            join[((wave * JF + j) * 4 + x) * 64 + lane] =
                Acc4{acc[j][4 * x], acc[j][4 * x + 1], acc[j][4 * x + 2], acc[j][4 * x + 3]};
    __syncthreads();
    Acc4 z[2] = {};
#pragma unroll
    for (int j = 0; j < JF; j++) {
        z[j] = join[(j * 4 + wave) * 64 + lane];
#pragma unroll
        for (int w = 1; w < kWaves; w++) z[j] += join[((w * JF + j) * 4 + wave) * 64 + lane];
    }
    switch (g.act) {
        case kActRelu: skinny_store<P, kActRelu, GATED>(g, td, o0, cols, z[0], z[1]); break;
        case kActSilu: skinny_store<P, kActSilu, GATED>(g, td, o0, cols, z[0], z[1]); break;
        case kActGelu: skinny_store<P, kActGelu, GATED>(g, td, o0, cols, z[0], z[1]); break;
        default: skinny_store<P, kActNone, GATED>(g, td, o0, cols, z[0], z[1]);
    }
}

template <typename P, typename SH>
hipError_t launch_shape(const GroupedGemmArgs& g, hipStream_t stream, LaunchInfo* info, bool run) {
    const int n_out = g.gated ? g.N / 2 : g.N;
    const int out_cols = g.gated ? SH::kBN / 2 : SH::kBN;
    // m segments that have rows, and do not overlap, hold at most m + (max_rows - m) / kBM
    // tiles. A tile that no segment has costs a workgroup that finds this out: with
    // max_rows / kBM + E tiles, 1 token through 2 of 8 int8 experts (K 4096, N 16384)
    // launched four times what it needed, 26.5 us instead of 24.2. The bf16 product's
    // interface does not exclude segments that overlap, so its grid has room for some.
    const int64_t m = g.E < g.max_rows ? g.E : g.max_rows;
    const int64_t max_tiles = P::kScaled ? m + (g.max_rows - m) / SH::kBM
                                         : (g.max_rows + SH::kBM - 1) / SH::kBM + g.E;
    const int64_t items = max_tiles * ((n_out + out_cols - 1) / out_cols);
    const int64_t grid = (items + kXcds - 1) / kXcds * kXcds;
    constexpr bool kSkinny = SH::kBN <= 64;
    constexpr bool kStreamed = [] {
        if constexpr (kSkinny) return SH::kStream;
        else return false;
    }();
    if (info)
        *info = LaunchInfo{grid, SH::kThreads, (size_t)SH::kLds, SH::kBM,
                           kStreamed ? P::kStreamedName : P::kName};
    if (!run) return hipSuccess;
    const dim3 blocks((unsigned)grid), threads(SH::kThreads);
    if constexpr (kSkinny) {
        if constexpr (SH::kBN == 64) {
            if (g.gated) k_grouped_gemm_skinny<P, SH, true><<<blocks, threads, 0, stream>>>(g);
            else k_grouped_gemm_skinny<P, SH, false><<<blocks, threads, 0, stream>>>(g);
        } else {
            k_grouped_gemm_skinny<P, SH, false><<<blocks, threads, 0, stream>>>(g);
        }
    } else {
        if (g.gated) k_grouped_gemm<P, SH, true><<<blocks, threads, 0, stream>>>(g);
        else k_grouped_gemm<P, SH, false><<<blocks, threads, 0, stream>>>(g);
    }
    return hipGetLastError();
}

}  // namespace

}  // namespace moe
