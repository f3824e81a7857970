// Launch interface of the norms around a block (residual_norm.cu) for the host
// code (host_linear.cu).  Not part of the public C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mbert {

constexpr int kResidualNormMaxWidth = 16384;    // 16 warps with 32 numbers a lane

struct ResidualNormArgs {
    const void *x = nullptr, *branch = nullptr, *gate = nullptr;
    const void *weight = nullptr, *bias = nullptr;              // of y's norm; null weight: no y
    const void *after_weight = nullptr, *after_bias = nullptr;  // of the branch's; null weight: none
    void *h = nullptr, *y = nullptr;
    long long x_row = 0, branch_row = 0, gate_row = 0, h_row = 0, y_row = 0;    // strides in elements
    const int32_t *cu = nullptr;        // the sequences that rows of `gate` belong to
    int n_seqs = 0;
    long long rows = 0;
    int width = 0;
    int vectors = 0;                    // every row is of whole, 16-byte aligned vectors
    float residual_scale = 1.f, eps = 0.f;
    // the sum of numbers times sum_scale (a power of two, 1 / width or less), times
    // half_mean_scale: half their mean
    float sum_scale = 1.f, half_mean_scale = 0.5f, inv_width = 1.f;
    // squares that add up to less than this have the row scaled by 2^most_scale at most
    float least_squares = 0.f;
    int most_scale = 0;
    int32_t *err = nullptr;
    int gate_channels = 0;              // one gate for all rows
    // set by the launcher: lanes of a row, or warps of 32; the ring's slots, a row's bytes
    // there, the tensors whose rows a slot holds
    int lanes = 32, warps = 1, slots = 1, row_bytes = 0, tensors = 1;
};

cudaError_t launch_residual_norm(ResidualNormArgs &a, int dtype, bool layer, int num_sms, cudaStream_t stream);

}  // namespace mbert
