// Internal launchers shared by the C ABI (api.hip) and the kernel files.
// Arguments are assumed validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// Largest expert count the kernels accept (MOE_MAX_EXPERTS of the C ABI).
constexpr int kMaxExperts = 1024;

struct LaunchInfo {
    int64_t grid = 0;
    int block = 0;
    size_t lds = 0;
    int64_t param = 0;           // kernel-specific: lanes per token, tokens per block, ...
    const char* name = nullptr;  // for the launch log
};

// A launch packet counts work-items in 32 bits (grid_size_x) and blocks in
// 31: a kernel fits when blocks * threads < 2^32 and blocks < 2^31.
inline bool launch_fits(const LaunchInfo& i) {
    return i.grid >= 0 && i.grid < ((int64_t)1 << 31) &&
           i.grid * (int64_t)i.block < ((int64_t)1 << 32);
}

// Every launcher below fills `info` (one entry per kernel it enqueues, in
// order) before launching anything; with run == false it only fills `info`,
// so callers can check the geometry of a whole call before the first launch.

hipError_t launch_route_topk(const float* logits, int64_t T, int E, int k, int n_shared,
                             float shared_w, int32_t* topk_idx, float* topk_w,
                             hipStream_t stream, LaunchInfo* info, bool run = true);

hipError_t launch_route_replicas(int32_t* topk_idx, int64_t T, int k, int E,
                                 const int32_t* replica_base, hipStream_t stream);

struct DispatchArgs {
    const void* x;
    const int32_t* topk_idx;     // routing table; written here first when logits != nullptr
    const float* logits;         // [T, E]: route inside the dispatch (moe_route_dispatch), or nullptr
    float* topk_w;               // [T, k] router weights out, with logits
    int64_t T;
    int H, E, k, groups, row_align;
    bool fp8;
    void* out;
    float* out_scales;
    int32_t* expert_counts;
    int32_t* expert_offsets;
    int32_t* group_offsets;
    int32_t* row_src;
    int32_t* dst_row;
    uint8_t* tile_counts;   // workspace [tiles, E]
    int32_t* tile_base;     // workspace [tiles, E]
    uint8_t* tile_rank;     // workspace [T, k]
    int64_t max_rows;       // rows in out / out_scales / row_src
    // moe_dispatch_quantized: x and out are rows of 2 H bytes with `scales` scales each
    const float* x_scales = nullptr;   // [T, scales]
    int scales = 0;
};

// Tokens per count tile (16, 32 or 64, growing with T; at most 64, so tile
// counts and in-tile ranks fit a byte) and the tile count.
int dispatch_tile_tokens(int64_t T);
int64_t dispatch_tiles(int64_t T);

// Workspace layout (each part 256-byte aligned): byte tile counts
// [tiles, E] at counts_off, tile prefixes int32 [tiles, E] at base_off, byte
// in-tile ranks [T, k] at rank_off; total bytes. Nothing is kept between
// calls.
struct DispatchWorkspace {
    int tile_tokens;
    int64_t tiles;
    size_t counts_off, base_off, rank_off, total;
};
DispatchWorkspace dispatch_workspace(int64_t T, int E, int k);

// Up to four kernels: [route (only when routing falls back to its own
// kernel)], count (with routing inside when it applies), [scan (small
// batches scan inside the scatter)], scatter. *n gets the number of kernels.
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t stream, LaunchInfo info[4], int* n,
                           bool run = true);

// Rows already quantised (scales > 0), at most kDirectPairs slots that are not too many
// for their experts: one kernel that needs no workspace.
constexpr int64_t kDirectPairs = 32768;
bool dispatch_direct_applies(int64_t T, int E, int k);
hipError_t launch_dispatch_direct(const DispatchArgs& a, hipStream_t stream, LaunchInfo* info,
                                  bool run = true);

hipError_t launch_combine(const void* expert_out, const int32_t* dst_row, const float* topk_w,
                          int64_t T, int H, int k, void* y, hipStream_t stream,
                          LaunchInfo* info, bool run = true);

hipError_t launch_combine_send(const void* expert_out, const int32_t* dst_row,
                               const float* topk_w, const int32_t* topk_idx, int64_t T, int H,
                               int E, int k, int groups, void* partial, int32_t* count,
                               hipStream_t stream, LaunchInfo* info, bool run = true);

hipError_t launch_combine_recv(const void* partial, const int32_t* count, int64_t T, int H,
                               int k, void* y, hipStream_t stream, LaunchInfo* info,
                               bool run = true);

hipError_t launch_expert_scale(const void* disp, const float* disp_scales,
                               const int32_t* row_src, const int32_t* topk_idx,
                               const int32_t* expert_offsets, int64_t max_rows, int H,
                               int E, bool fp8, bool identity, void* expert_out,
                               hipStream_t stream);

// Grouped GEMM: tile-list workspace size and launcher (tile list + GEMM).
size_t gemm_workspace_bytes(int64_t max_rows, int E);
int64_t gemm_max_tiles(int64_t max_rows, int E);
hipError_t launch_grouped_gemm_fp8(const void* a, const float* a_scales,
                                   const int32_t* expert_offsets, const void* w,
                                   const float* w_scales, int E, int N, int K, int64_t max_rows,
                                   void* y, void* workspace, hipStream_t stream,
                                   LaunchInfo info[2], bool run = true);

// Scored router gate (moe_route_scored).
struct ScoredArgs {
    const void* logits;          // [T, E], rows ld apart; fp32 or bf16
    const float* bias;           // [E] or nullptr
    int32_t* topk_idx;
    float* topk_w;
    int64_t T, ld;
    int E, k, n_group, topk_group, group_top, n_shared;
    float scale, shared_w;
    bool bf16, sigmoid, renorm;
};
hipError_t launch_route_scored(const ScoredArgs& a, hipStream_t stream, LaunchInfo* info,
                               bool run = true);

// Grouped GEMMs with an epilogue (moe_grouped_gemm_bf16, moe_grouped_gemm_int8).
// Operand rows are K 2-byte units: bf16 values, or pairs of int8 values.
struct GroupedGemmArgs {
    const uint16_t* a;
    const int32_t* off;
    const uint16_t* w;
    const uint16_t* bias;        // [E, N] or nullptr
    const uint16_t* residual;    // [max_rows, N or N/2] or nullptr
    uint16_t* y;
    const float* a_scales;       // int8: [max_rows]
    const float* w_scales;       // int8: [E, N]
    int64_t max_rows;
    int E, N, K, act;
    bool gated;
};
hipError_t launch_grouped_gemm_bf16(const GroupedGemmArgs& g, hipStream_t stream, LaunchInfo* info,
                                    bool run = true);
hipError_t launch_grouped_gemm_int8(const GroupedGemmArgs& g, hipStream_t stream, LaunchInfo* info,
                                    bool run = true);

// Residual, root-mean-square norm and 8-bit output (moe_rmsnorm_quant).
struct NormArgs {
    const uint16_t* x;           // rows ld apart
    const uint16_t* residual;    // or nullptr
    const uint16_t* weight;
    uint16_t* sum;               // or nullptr
    uint16_t* y;                 // or nullptr
    uint8_t* out;
    float* scales;
    int64_t T, ld;
    int H;
    float eps, inv_h;            // 1 / H
    bool fp8;
};
hipError_t launch_rmsnorm_quant(const NormArgs& a, hipStream_t stream, LaunchInfo* info,
                                bool run = true);

// Gated activation with INT8 quantisation (moe_gated_act_quant_int8).
hipError_t launch_gated_act_int8(const void* h, const int32_t* expert_offsets, int E,
                                 int64_t max_rows, int I, int act, void* out, float* out_scales,
                                 hipStream_t stream, LaunchInfo* info, bool run = true);

// Gated activation with FP8 quantisation (moe_gated_act_quant_fp8).
hipError_t launch_gated_act_fp8(const void* h, const int32_t* expert_offsets, int E,
                                int64_t max_rows, int I, int act, void* out, float* out_scales,
                                hipStream_t stream, LaunchInfo* info, bool run = true);

}  // namespace moe
