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

hipError_t launch_grouped_gemm_int8(const GroupedGemmArgs& g, hipStream_t stream, LaunchInfo* info,
                                    bool run) {
    const int64_t hit = g.E < g.max_rows ? g.E : g.max_rows;
    const double r = hit ? (double)g.max_rows / hit : 0.0;
    if (r <= 32.0)
        return g.K % 64 == 0 ? launch_shape<Int8, Skinny<true>>(g, stream, info, run)
                             : launch_shape<Int8, Skinny<false>>(g, stream, info, run);
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
        return launch_shape<Int8, Large>(g, stream, info, run);
    if (medium <= small && medium <= skinny) return launch_shape<Int8, Medium>(g, stream, info, run);
    if (small <= skinny) return launch_shape<Int8, Small>(g, stream, info, run);
    return launch_shape<Int8, Skinny<false>>(g, stream, info, run);
}

}  // namespace moe
