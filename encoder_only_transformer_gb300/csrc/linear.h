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
    CUtensorMap tm_out, tm_residual;    // [rows][outer], box 64 columns x 32 rows (linear.cu, where
                                        // out_tma / residual_tma say that the rows allow it)
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
    int bias_vectors = 0;               // bias at n (and outer + n) is 16-byte aligned for n % 8 == 0
    int out_tma = 0, residual_tma = 0;
    int32_t *err = nullptr;
};

// The kernel for many rows: a pair of SMs per 256 rows x `columns` (128 or 256)
// accumulator columns, half as many output columns where gated.
constexpr int kLinearRows = 256;
cudaError_t launch_linear(const LinearArgs &a, int columns, bool gated, bool half, long long units, int num_sms,
                          cudaStream_t stream);

// The kernel for few rows: 128 output columns x `tile` rows (16, 32, 64 or 128),
// the inner dimension shared by `split` CTAs of a cluster.  With split > 1 a
// unit has a cluster of its own.
constexpr int kLinearRowsColumns = 128;
// the split of `tile` rows is at most this (what fits in shared memory beside the ring)
constexpr int linear_rows_most_split(int tile, bool gated) { return tile == 128 && gated ? 1 : 8; }
// CTAs on one SM
constexpr int linear_rows_ctas(int tile, bool gated) { return gated && tile >= 64 ? 1 : 2; }
cudaError_t launch_linear_rows(const LinearArgs &a, int tile, int split, bool gated, bool half, long long units,
                               int num_sms, cudaStream_t stream);

}  // namespace mbert
