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
// Work split: segments are cut into row tiles; a workgroup finds its tile by a
// scan over the segment lengths (no list kernel, no workspace). Tile shapes
// from 256 x 256 to 32 x 64 and the rule between them stand at the launcher.
// Operands go from memory straight into LDS (buffer_load ... lds) and are
// multiplied by v_mfma_f32_32x32x16_bf16 into fp32 accumulators. In the gated
// form a wave's weight rows are half gate, half up of the same output columns,
// so the product is formed lane by lane.
//
// Many rows: bound by the matrix cores, in practice by the clock they run at.
// With 16 experts of 1024 rows, N 4096 (gated), K 7168: 777 us, 1240 TFLOP/s;
// 16384 x 4096 x 7232: 708 us, 1370 TFLOP/s, where the library's plain product
// of that size runs at 1490. Both clock down to 1.5-1.7 GHz; the matrix cores
// are busy 70 % of the cycles. Steps that counted: LDS stages as separate
// arrays (else every read waits for all DMA: 13.4 -> 10.1 ms on 16384 tokens
// over 256 experts), row bands (L2 misses 33 -> 22 GB, 8.6 -> 7.9 ms), a third
// weight stage (7.4 ms), four waves of 128 x 128 instead of eight of 128 x 64
// with the DMA spread over the products (7.1-7.3 ms; a third fewer LDS reads).
// Few rows: bound by the weights, see the skinny kernel.
#include "grouped_gemm_tile.h"

namespace moe {

// The shape of a call, from what the host knows: the capacity, from which the
// rows of an expert that has any, r (with padded segments more than there are).
//
// r <= 32: Skinny, whose tile holds a segment of average length, so that segments
// of like length read their weights once. A longer one reads them again: 256
// experts, K 7168, N 4096 (gated), ragged segments of mean r, us:
//   r           4     8    12    16    24    32
//   Skinny   2000  2136  2198  2308  2910  3575
//   Medium   2291  2363  2374  2385  2417  2495
// For such segments the border would be better at about 18; the host does not know
// how ragged they are. With rows of whole 128-byte lines (K % 64 == 0) the weights
// are streamed: r = 4 above is 2000 us (7.4 TB/s), 2261 us without the hint. Lines
// shared by two k-blocks would be fetched twice (18 tokens, K 2200: 49 us streamed,
// 38 us not).
//
// Otherwise the shape of least estimated time: rounds of the chip times the
// time of a round, start + k-blocks times a rate (us), fitted to:
//   us, experts x rows, N, K           Large  Medium  Small  Skinny
//   16 x 400, 4096, 2048                121     133    148     383
//    8 x 1000, 4096, 4096               219     265    290     834
//   55 x 286, 2336, 392                 123      95     85     233
//   37 x 480, 2352, 144                  73      57     54     230
//    1 x 2048, 4096, 4096                84      65     66     199
//   12 x 194, 1032, 1016                 27      20     16      29
//    1 x 128, 4096, 4096                 70      41     35      20
//    5 x 217, 416, 4584                  84      66     46      23
// A segment ends inside a tile, half a tile on average; a lone segment's tiles
// are known. The last round counts a quarter more than its share. Padded segments
// of few tokens count as their capacity (one token through 8 of 256 experts, 128-row
// segments, K 7168, N 4096: Medium 126 us, Small 127, Skinny, whose grid over the
// capacity has 163 thousand workgroups, 422).
hipError_t launch_grouped_gemm_bf16(const GroupedGemmArgs& g, hipStream_t stream, LaunchInfo* info,
                                    bool run) {
    const int64_t hit = g.E < g.max_rows ? g.E : g.max_rows;
    const double r = hit ? (double)g.max_rows / hit : 0.0;
    if (r <= 32.0)
        return g.K % 64 == 0 ? launch_shape<Bf16, Skinny<true>>(g, stream, info, run)
                             : launch_shape<Bf16, Skinny<false>>(g, stream, info, run);
    const double kb = (g.K + kBK - 1) / kBK;
    auto items = [&](int bm, int bn) {
        double per = r / bm + 0.5;
        if (hit == 1) per = (double)((g.max_rows + bm - 1) / bm);
        return hit * (per > 1.0 ? per : 1.0) * ((g.N + bn - 1) / bn);
    };
    auto rounds = [](double n, int slots) { return n <= slots ? 1.0 : n / slots + 0.25; };
    const double small_n = items(128, 128), skinny_n = items(32, 64);
    const double large = rounds(items(256, 256), 256) * (12.0 + 1.6 * kb);
    const double medium = rounds(items(128, 256), 256) * (8.0 + 1.0 * kb);
    const double small = small_n <= 256 ? 5.0 + 0.55 * kb : rounds(small_n, 512) * (6.0 + 1.1 * kb);
    const double skinny = skinny_n <= 256 ? 2.0 + 0.23 * kb : rounds(skinny_n, 512) * (3.0 + 0.4 * kb);
    if (large <= medium && large <= small && large <= skinny)
        return launch_shape<Bf16, Large>(g, stream, info, run);
    if (medium <= small && medium <= skinny) return launch_shape<Bf16, Medium>(g, stream, info, run);
    if (small <= skinny) return launch_shape<Bf16, Small>(g, stream, info, run);
    return launch_shape<Bf16, Skinny<false>>(g, stream, info, run);
}

}  // namespace moe
