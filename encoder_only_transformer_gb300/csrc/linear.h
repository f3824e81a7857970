// Launch interface of the products of any width (linear.cu, linear_rows.cu) for
// the host code (host_linear.cu).  Not part of the public C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mbert {

// out = residual + scale act(x W^T + b), or gated, with W = [Wg; Wu]:
// residual + scale act(x Wg^T + bg) (x Wu^T + bu); rows in groups (experts),
// each with a W and b of its own, or all in one.
struct LinearArgs {
    CUtensorMap tm_x;                   // [rows][inner], box 64 columns
    CUtensorMap tm_w;                   // [groups][width][inner], box 64 columns, one group
    CUtensorMap tm_out, tm_residual;    // [rows][outer], box linear_chunk columns x 32 rows (linear.cu, where
                                        // out_vectors / residual_vectors say that the rows allow it)
    const void *bias = nullptr;         // [groups][width]
    const void *residual = nullptr;
    const float *row_scale = nullptr;
    void *out = nullptr;
    long long residual_row = 0, out_row = 0;    // row strides in elements
    const int32_t *cu = nullptr;        // [groups + 1]; null: one group of all rows
    int groups = 1;
    long long rows = 0;
    int inner = 0, outer = 0;
    int activation = 0;                 // MBERT_ACT_*
    // linear_rows.cu: granules of a piece, stages of its ring, bytes of one
    int granules = 0, stages = 0, stage_bytes = 0;
    int out_vectors = 0, residual_vectors = 0;
    int out_bytes = 2, residual_bytes = 2;      // else: bytes of a word, 2, 4 or 8
    int32_t *err = nullptr;
};

// The kernel for many rows: a pair of SMs per 256 rows x `columns` (128 or 256)
// accumulator columns, half as many output columns where gated.
constexpr int kLinearRows = 256;
constexpr int linear_chunk(bool gated) { return gated ? 64 : 32; }  // output columns of its staging buffers
cudaError_t launch_linear(const LinearArgs &a, int columns, bool gated, bool half, long long units, int num_sms,
                          cudaStream_t stream);

// The kernel for few rows: `tile` rows (16, 32, 64 or 128) x up to `granules` times 32
// output columns a piece, the inner dimension shared by `split` CTAs of a cluster.
// The pieces of all row tiles are dealt out evenly to `ctas` CTAs; with a split every
// piece has a cluster of its own, `ctas` of them.
constexpr int kLinearGranule = 32;
constexpr int kLinearGranules = 4;      // at most
struct LinearRowsPlan {
    int tile, granules, split;
    long long ctas;
};
// CTAs on one SM, the shared memory of one
constexpr int linear_rows_ctas(int tile, bool gated) { return tile * (gated ? 2 : 1) >= 128 ? 1 : 2; }
constexpr int linear_rows_budget(int tile, bool gated) { return linear_rows_ctas(tile, gated) == 2 ? 112 * 1024 : 224 * 1024; }
constexpr int kLinearRowsFixed = 10 * 1024;     // of it beside the ring and the parts of sums
constexpr int kLinearRowsStages = 24;           // at most
// bytes of the sums that the CTAs of a cluster exchange, of a stage of the ring; its stages
constexpr int linear_rows_parts(int tile, bool gated, int granules, int split)
{
    return split > 1 ? (gated ? 2 : 1) * tile * granules * kLinearGranule * 4 : 0;
}
constexpr int linear_rows_stage(int tile, bool gated, int granules)
{
    return tile * 128 + (gated ? 2 : 1) * granules * kLinearGranule * 128;
}
constexpr int linear_rows_stages(int tile, bool gated, int granules, int split)
{
    const int left = linear_rows_budget(tile, gated) - kLinearRowsFixed - linear_rows_parts(tile, gated, granules, split) -
                     (kLinearGranules - granules) * kLinearGranule * 128;
    const int n = left / linear_rows_stage(tile, gated, granules);
    return n < kLinearRowsStages ? n : kLinearRowsStages;
}
cudaError_t launch_linear_rows(const LinearArgs &a, const LinearRowsPlan &p, bool gated, bool half, cudaStream_t stream);

// How a product runs: the kernel for few rows, or that of `columns` accumulator columns
// and at most `units` of them.
struct LinearPlan {
    bool few;
    LinearRowsPlan rows;
    int columns;
    long long units;
};

// A plan and the sizes that it is for.
struct PlanEntry {
    bool known = false;
    int64_t key[4] = {};
    LinearPlan plan = {};
};

}  // namespace mbert
