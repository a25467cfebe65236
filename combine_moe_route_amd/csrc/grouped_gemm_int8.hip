// Grouped INT8 GEMM over segments of quantised rows, with one scale a row and one
// a weight channel, bias, activation, gating and residual in the epilogue.
//
// Expert e owns rows [off[e], off[e+1]) of a. With the whole-number sum
// t[n] = sum_k a[r, k] w[e, n, k] (exact in 32 bits: K <= 2^17 - 16) and
//
//   z[n] = fp32(t[n]) * a_scales[r] * w_scales[e, n] + bias[e, n]
//
// the rest is the bf16 product's: y = act(z) + residual, or gated
// y = act(z[:, :N/2]) * z[:, N/2:] + residual, rounded once to bf16.
#include "grouped_gemm_tile.h"

namespace moe {

// Skinny tiles of 64 weight rows, or of 32 where those would leave half of the chip
// idle: a CU takes in no more than about 35 GB/s here, whatever is in flight (twice
// the waves a workgroup changed nothing). 16 rows, K 7168, N 2400: 17.5 -> 12.9 us;
// one row, K 2048, N 7168: 8.1 -> 6.7; K 130000, N 64: 148 -> 98; but with 256 tiles
// of 64, 128 rows, K 8192, N 4096: 18.6 -> 24.5.
static hipError_t launch_skinny(const GroupedGemmArgs& g, double tiles, bool streamed,
                                hipStream_t stream, LaunchInfo* info, bool run) {
    if (tiles <= 128.0 && !g.gated)
        return streamed ? launch_shape<Int8, Skinny<true, 32>>(g, stream, info, run)
                        : launch_shape<Int8, Skinny<false, 32>>(g, stream, info, run);
    return streamed ? launch_shape<Int8, Skinny<true>>(g, stream, info, run)
                    : launch_shape<Int8, Skinny<false>>(g, stream, info, run);
}

// The shape of a call, from what the host knows: the capacity, from which the
// rows of an expert that has any, r (with padded segments more than there are).
//
// r <= 20: Skinny, whose tile holds a segment of average length. Segments longer than
// its 32 rows read their weights again: 256 experts, K 7168, N 4096, ragged segments
// of mean r, us:
//   r                   4     8    16    24    32    48
//   Skinny           1060  1110  1183  1358  1924  2679
//   Medium           1187  1218  1241  1259  1277  1306
// With rows of whole 128-byte lines (K % 128 == 0) the weights are streamed with the
// non-temporal hint (7.3 TB/s at r = 4; without it 1167 us). Lines that two k-blocks
// share would be fetched twice.
//
// Otherwise the shape of least estimated time: rounds of the chip times the time of a
// round, start + k-blocks times a rate that grows with the share of the chip that is
// busy (us). Measured, experts x rows, K, N (* the choice):
//                          Large  Medium  Small  Skinny
//   16 x 400, 4096, 4096    132*    143    157     423
//    8 x 1000, 8192, 4096   235*    281    308     894
//   16 x 1024, 7168, 4096   425*    528    574    1571
//    1 x 2048, 8192, 4096    77      66*    68     196
//   55 x 286, 784, 2336     119      99     94*    242
//   37 x 480, 288, 2352      62      54     54*    199
//   12 x 194, 2032, 1032     30      20     17*     29
//   20 x 450, 3600, 904      48*     57     61     117
//    1 x 128, 8192, 4096     72      40     34      19*
//    5 x 217, 9168, 416      82      61     45      23*
// A segment ends inside a tile, half a tile on average; a lone segment's tiles are
// known. The last round counts a quarter more than its share. Skinny is for launches
// that it fits on the chip in one round: with more, its estimate misses that weights
// are read again.
hipError_t launch_grouped_gemm_int8(const GroupedGemmArgs& g, hipStream_t stream, LaunchInfo* info,
                                    bool run) {
    const int64_t hit = g.E < g.max_rows ? g.E : g.max_rows;
    const double r = hit ? (double)g.max_rows / hit : 0.0;
    const double kb = (g.K + kBK - 1) / kBK;
    auto items = [&](int bm, int bn) {
        double per = r / bm + 0.5;
        if (hit == 1) per = (double)((g.max_rows + bm - 1) / bm);
        return hit * (per > 1.0 ? per : 1.0) * ((g.N + bn - 1) / bn);
    };
    auto rounds = [](double n, int slots) { return n <= slots ? 1.0 : n / slots + 0.25; };
    auto busy = [](double n) { return n < 256 ? n / 256 : 1.0; };
    const double skinny_n = items(32, 64);
    if (r <= 20.0) return launch_skinny(g, skinny_n, g.K % kBK == 0, stream, info, run);
    const double large_n = items(256, 256), medium_n = items(128, 256), small_n = items(128, 128);
    const double large = rounds(large_n, 256) * (12.0 + (1.0 + 0.6 * busy(large_n)) * kb);
    const double medium = rounds(medium_n, 256) * (8.0 + (0.65 + 0.35 * busy(medium_n)) * kb);
    const double small = small_n <= 256 ? 5.0 + 0.55 * kb : rounds(small_n, 512) * (6.0 + 1.1 * kb);
    const double skinny = skinny_n <= 256   ? 2.0 + 0.23 * kb
                          : skinny_n <= 512 ? 3.0 + 0.4 * kb
                                            : 1e30;
    if (large <= medium && large <= small && large <= skinny)
        return launch_shape<Int8, Large>(g, stream, info, run);
    if (medium <= small && medium <= skinny) return launch_shape<Int8, Medium>(g, stream, info, run);
    if (small <= skinny) return launch_shape<Int8, Small>(g, stream, info, run);
    return launch_skinny(g, skinny_n, false, stream, info, run);
}

}  // namespace moe
