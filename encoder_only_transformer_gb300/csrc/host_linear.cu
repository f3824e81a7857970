// Host side of the products of any width and of the norms around a block: argument
// checks, tensor maps, the choice of the kernel.
#include <algorithm>
#include <cmath>

#include "mbert_attn.h"
#include "common.cuh"
#include "handle.h"
#include "internal.h"
#include "linear.h"
#include "residual_norm.h"

#define MBERT_API extern "C" __attribute__((visibility("default")))

using namespace mbert;

namespace {

constexpr int64_t kMaxRows = INT32_MAX - 1024;
constexpr int kMaxWidth = 1 << 24;
// Elements from a tensor's first to its last, at most: beyond any device's memory,
// and far from where extents in bytes would overflow.
constexpr int64_t kMaxSpan = 1ll << 48;

// Rows of `width` elements, `pitch` elements apart.
struct Rows {
    const void *p;
    int64_t rows, pitch, width;
    int es;

    bool ok() const
    {
        return p && reinterpret_cast<uintptr_t>(p) % es == 0 &&
               (rows <= 1 || (pitch >= width && pitch <= kMaxSpan / rows)) && width <= kMaxSpan;
    }
    uintptr_t lo() const { return reinterpret_cast<uintptr_t>(p); }
    uintptr_t hi() const { return lo() + static_cast<uintptr_t>(((rows - 1) * pitch + width) * es); }
    bool aligned(int bytes) const { return lo() % bytes == 0 && (rows <= 1 || pitch * es % bytes == 0); }
    bool none() const { return !p || rows <= 0 || width <= 0; }
};

Rows flat(const void *p, int64_t n, int es) { return {p, 1, n, n, es}; }

// May some element of a be an element of b?  Exact where both have the same pitch
// (column blocks of the same rows); else by extent.
bool meet(const Rows &a, const Rows &b)
{
    if (a.none() || b.none() || a.hi() <= b.lo() || b.hi() <= a.lo())
        return false;
    if (a.rows <= 1 || b.rows <= 1 || a.pitch != b.pitch || a.es != b.es)
        return true;
    const uintptr_t pitch = static_cast<uintptr_t>(a.pitch) * a.es;
    const uintptr_t d = b.lo() >= a.lo() ? (b.lo() - a.lo()) % pitch : (pitch - (a.lo() - b.lo()) % pitch) % pitch;
    return !(d >= static_cast<uintptr_t>(a.width) * a.es && d + static_cast<uintptr_t>(b.width) * b.es <= pitch);
}

// `a` may also be `b` itself, element for element.
bool meet_unless_same(const Rows &a, const Rows &b)
{
    return !(a.p == b.p && (a.rows <= 1 || a.pitch == b.pitch)) && meet(a, b);
}

// 3-D map of 16-bit elements over [groups][rows][inner], box 64 x `box` x 1, 128-byte
// swizzle, out-of-range reads give 0.
int encode_groups(const mbert_attn *h, CUtensorMap *tm, const void *p, int64_t inner, int64_t rows, int64_t groups,
                  int64_t pitch, int64_t group_pitch, int box)
{
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(groups)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch) * 2, static_cast<cuuint64_t>(group_pitch) * 2};
    const cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(box), 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    const CUresult r = h->encode(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, boxes,
                                 ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MBERT_OK : MBERT_ERR_CUDA;
}

// How a product runs: the kernel, its tiles, an upper bound on its units.
struct LinearPlan {
    bool rows;          // the kernel for few rows
    int tile;           // rows of its tile; else accumulator columns of the pair kernel
    int split;          // CTAs that share the inner dimension
    int64_t units;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Blocks of `rows` rows over all groups, at most.
int64_t block_bound(const mbert_attn_linear_args &c, int rows)
{
    if (c.experts == 0)
        return ceil_div(c.rows, rows);
    return std::min<int64_t>(c.rows, c.rows / rows + c.experts);
}

LinearPlan linear_plan(const mbert_attn *h, const mbert_attn_linear_args &c)
{
    LinearPlan p;
    const int64_t groups = std::max(c.experts, 1);
    const int64_t mean = ceil_div(c.rows, groups);      // rows of a group
    p.split = 1;
    p.rows = mean <= 128;
    if (p.rows) {
        const int64_t want = c.experts == 0 ? mean : 2 * mean;
        p.tile = want <= 16 ? 16 : want <= 32 ? 32 : want <= 64 ? 64 : 128;
        p.units = block_bound(c, p.tile) * ceil_div(c.outer, kLinearRowsColumns);
        const int64_t places = static_cast<int64_t>(h->num_sms) * linear_rows_ctas(p.tile, c.gated);
        const int64_t steps = ceil_div(c.inner, 64);
        while (p.split < linear_rows_most_split(p.tile, c.gated) && 2 * p.split <= steps &&
               p.units * p.split * 2 <= places)
            p.split *= 2;
        return p;
    }
    const int64_t pairs = h->num_sms / 2;
    p.tile = 256;
    p.units = block_bound(c, kLinearRows) * ceil_div(c.outer, c.gated ? 128 : 256);
    if (p.units <= pairs / 2) {
        p.tile = 128;
        p.units = block_bound(c, kLinearRows) * ceil_div(c.outer, c.gated ? 64 : 128);
    }
    return p;
}

}  // namespace

MBERT_API int mbert_attn_linear(mbert_attn *h, const mbert_attn_linear_args *args, void *stream)
{
    if (!h || !args)
        return MBERT_ERR_BAD_ARG;
    const mbert_attn_linear_args &c = *args;
    if (c.dtype != MBERT_BF16 && c.dtype != MBERT_F16)
        return MBERT_ERR_UNSUPPORTED;
    if (c.rows < 0 || c.rows > kMaxRows || c.inner < 1 || c.inner > kMaxWidth || c.outer < 1 || c.outer > kMaxWidth ||
        c.activation < MBERT_ACT_NONE || c.activation > MBERT_ACT_RELU || (c.gated != 0 && c.gated != 1) ||
        c.experts < 0 || c.experts > 65536)
        return MBERT_ERR_BAD_ARG;
    // the router's weights go with experts, a residual with the plain product
    if (c.experts > 0 ? c.residual != nullptr : c.cu_experts || c.row_scale)
        return MBERT_ERR_BAD_ARG;
    if (c.rows == 0)
        return MBERT_OK;
    if (c.experts > 0 && (!c.cu_experts || reinterpret_cast<uintptr_t>(c.cu_experts) % 4))
        return MBERT_ERR_BAD_ARG;
    const int64_t groups = std::max(c.experts, 1), width = static_cast<int64_t>(c.gated ? 2 : 1) * c.outer;
    const Rows x{c.x, c.rows, c.x_row, c.inner, 2}, out{c.out, c.rows, c.out_row, c.outer, 2};
    const Rows weight{c.weight, width, c.weight_row, c.inner, 2};
    const Rows residual{c.residual, c.rows, c.residual_row, c.outer, 2};
    if (!x.ok() || !out.ok() || !weight.ok() || (c.residual && !residual.ok()))
        return MBERT_ERR_BAD_ARG;
    // what TMA can fetch: 16-byte aligned rows
    const int64_t matrix = (width - 1) * c.weight_row + c.inner;
    if (!x.aligned(16) || !weight.aligned(16) ||
        (groups > 1 && (c.weight_expert < matrix || c.weight_expert % 8 || c.weight_expert > kMaxSpan / groups)))
        return MBERT_ERR_BAD_ARG;
    const Rows bias = flat(c.bias, groups * width, 2), scale = flat(c.row_scale, c.rows, 4);
    const Rows weights = flat(c.weight, (groups - 1) * c.weight_expert + matrix, 2);
    const Rows cu = flat(c.cu_experts, groups + 1, 4);
    if ((c.bias && !bias.ok()) || (c.row_scale && !scale.ok()) || meet(out, x) || meet(out, weights) ||
        meet(out, bias) || meet(out, scale) || meet(out, cu) || meet_unless_same(out, residual))
        return MBERT_ERR_BAD_ARG;

    const LinearPlan p = linear_plan(h, c);
    if (p.units > INT32_MAX / 4)
        return MBERT_ERR_BAD_ARG;       // (more than any device holds)
    DeviceGuard g(h->device);
    LinearArgs a;
    // a dimension of one element has no stride that matters; a map wants one all the same
    auto pitch = [](int64_t rows, int64_t given, int64_t w) { return rows > 1 ? given : (w + 7) / 8 * 8; };
    const int64_t wrow = pitch(width, c.weight_row, c.inner);
    const int xbox = p.rows ? p.tile : kLinearRows / 2, wbox = p.rows ? kLinearRowsColumns : p.tile / 2;
    if (encode_rows(h, &a.tm_x, c.x, c.inner, c.rows, pitch(c.rows, c.x_row, c.inner), xbox, 256) != MBERT_OK ||
        encode_groups(h, &a.tm_w, c.weight, c.inner, width, groups, wrow, groups > 1 ? c.weight_expert : width * wrow,
                      wbox) != MBERT_OK)
        return MBERT_ERR_CUDA;
    a.out_tma = !p.rows && out.aligned(16);
    a.residual_tma = !p.rows && c.residual && residual.aligned(16);
    if ((a.out_tma && encode_rows(h, &a.tm_out, c.out, c.outer, c.rows, pitch(c.rows, c.out_row, c.outer), 32, 256) !=
                          MBERT_OK) ||
        (a.residual_tma && encode_rows(h, &a.tm_residual, c.residual, c.outer, c.rows,
                                       pitch(c.rows, c.residual_row, c.outer), 32, 256) != MBERT_OK))
        return MBERT_ERR_CUDA;
    a.bias = c.bias;
    a.residual = c.residual;
    a.row_scale = c.row_scale;
    a.out = c.out;
    a.residual_row = c.residual_row;
    a.out_row = c.out_row;
    a.cu = c.cu_experts;
    a.groups = static_cast<int>(groups);
    a.rows = c.rows;
    a.inner = c.inner;
    a.outer = c.outer;
    a.activation = c.activation;
    a.bias_vectors = c.bias && bias.aligned(16) && c.outer % 8 == 0;
    a.err = h->err;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool half = c.dtype == MBERT_F16;
    const cudaError_t e = p.rows ? launch_linear_rows(a, p.tile, p.split, c.gated, half, p.units, h->num_sms, st)
                                 : launch_linear(a, p.tile, c.gated, half, p.units, h->num_sms, st);
    h->launches += 1;
    return e == cudaSuccess ? MBERT_OK : MBERT_ERR_CUDA;
}

MBERT_API int mbert_attn_residual_norm(mbert_attn *h, const mbert_attn_residual_norm_args *args, void *stream)
{
    if (!h || !args)
        return MBERT_ERR_BAD_ARG;
    const mbert_attn_residual_norm_args &c = *args;
    if (c.dtype < MBERT_BF16 || c.dtype > MBERT_F32 || c.rows < 0 || c.rows > kMaxRows || c.width < 1 ||
        c.width > kResidualNormMaxWidth || (c.norm != MBERT_NORM_RMS && c.norm != MBERT_NORM_LAYER) ||
        !(c.eps >= 0.f) || c.eps > 1.f || !std::isfinite(c.residual_scale))
        return MBERT_ERR_BAD_ARG;
    // a norm's bias with its weight; without a branch nothing is scaled or gated, and
    // the call is y's norm alone
    if ((c.bias && !c.weight) || (c.branch_bias && !c.branch_weight) || (c.cu_seqlens && !c.gate) ||
        (!c.branch && (c.branch_weight || c.gate || c.h || c.residual_scale != 1.f || !c.weight)) ||
        c.gate_kind < MBERT_GATE_NONE || c.gate_kind > MBERT_GATE_SEQUENCES ||
        (c.gate != nullptr) != (c.gate_kind != MBERT_GATE_NONE) ||
        (c.cu_seqlens != nullptr) != (c.gate_kind == MBERT_GATE_SEQUENCES) || (c.cu_seqlens && c.n_seqs < 1) ||
        reinterpret_cast<uintptr_t>(c.cu_seqlens) % 4)
        return MBERT_ERR_BAD_ARG;
    if (c.rows == 0)
        return MBERT_OK;
    const int es = c.dtype == MBERT_F32 ? 4 : 2;
    const int64_t gates = c.gate_kind == MBERT_GATE_ROWS ? c.rows : c.gate_kind == MBERT_GATE_SEQUENCES ? c.n_seqs : 1;
    const Rows x{c.x, c.rows, c.x_row, c.width, es}, branch{c.branch, c.rows, c.branch_row, c.width, es};
    const Rows gate{c.gate, gates, c.gate_row, c.width, es};
    const Rows hr{c.h, c.rows, c.h_row, c.width, es}, y{c.y, c.rows, c.y_row, c.width, es};
    if (!x.ok() || (c.branch && (!branch.ok() || !hr.ok())) || (c.gate && !gate.ok()) || (c.weight && !y.ok()))
        return MBERT_ERR_BAD_ARG;
    const Rows cu = flat(c.cu_seqlens, static_cast<int64_t>(c.n_seqs) + 1, 4);
    const void *const params[4] = {c.weight, c.bias, c.branch_weight, c.branch_bias};
    bool vectors = c.width * es % 16 == 0;
    for (const Rows *r : {&x, &branch, &gate, &hr, &y})
        vectors = vectors && (r->none() || r->aligned(16));
    for (const void *p : params) {
        const Rows r = flat(p, c.width, es);
        if (p && (!r.ok() || (c.branch && meet(hr, r)) || (c.weight && meet(y, r))))
            return MBERT_ERR_BAD_ARG;
        vectors = vectors && reinterpret_cast<uintptr_t>(p) % 16 == 0;
    }
    // h may be x or the branch, and so may y; no two results share elements
    for (const Rows *r : {&hr, &y}) {
        if (r == &hr ? !c.branch : !c.weight)
            continue;
        if (meet_unless_same(*r, x) || meet_unless_same(*r, branch) || meet(*r, gate) || meet(*r, cu))
            return MBERT_ERR_BAD_ARG;
    }
    if (c.branch && c.weight && meet(hr, y))
        return MBERT_ERR_BAD_ARG;

    ResidualNormArgs a;
    a.x = c.x;
    a.branch = c.branch;
    a.gate = c.gate;
    a.weight = c.weight;
    a.bias = c.bias;
    a.after_weight = c.branch_weight;
    a.after_bias = c.branch_bias;
    a.h = c.h;
    a.y = c.y;
    a.x_row = c.x_row;
    a.branch_row = c.branch_row;
    a.gate_row = c.gate_row;
    a.gate_channels = c.gate_kind == MBERT_GATE_CHANNELS;
    a.h_row = c.h_row;
    a.y_row = c.y_row;
    a.cu = c.cu_seqlens;
    a.n_seqs = c.n_seqs;
    a.rows = c.rows;
    a.width = c.width;
    a.vectors = vectors;
    a.residual_scale = c.residual_scale;
    a.eps = c.eps;
    int k = 0;
    while ((1 << k) < c.width)
        ++k;
    a.sum_scale = std::ldexp(1.f, -k);
    a.half_mean_scale = static_cast<float>(std::ldexp(0.5, k) / c.width);
    a.inv_width = static_cast<float>(1.0 / c.width);
    a.least_squares = c.eps >= 0x1p-40f ? 0.f : 0x1p-90f;
    a.most_scale = c.eps > 0.f ? std::min(126, (100 - std::ilogb(c.eps)) / 2) : 126;
    a.err = h->err;
    DeviceGuard g(h->device);
    const cudaError_t e = launch_residual_norm(a, c.dtype, c.norm == MBERT_NORM_LAYER, h->num_sms,
                                               static_cast<cudaStream_t>(stream));
    h->launches += 1;
    return e == cudaSuccess ? MBERT_OK : MBERT_ERR_CUDA;
}
